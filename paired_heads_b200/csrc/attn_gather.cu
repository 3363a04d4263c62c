// attn_gather.cu -- bf16 attention on the sm_100a tensor cores over gathered keys: causal with a
// sliding window and sinks, keys in packed documents or in the pages of a cache.
//
// Mathematics: o = softmax(scale q k^T) v row by row over the visible key columns (gather.cuh), one
// pass with a running maximum and sum; an item that a cut between two CTAs' shares divides leaves
// normalised partial rows and their log-sum-exp, two places a CTA, for attn_join_cuts_kernel.
//
// A row tile is up to 256 rows, two sub-tiles of 128: `pack` query heads of one kv head's group times
// tile_tokens tokens. Packing the group multiplies the rows that each loaded key tile serves and lets
// a few new tokens fill the M = 128 of the MMA. The key columns come in tiles of 128. Tiles of plain
// window columns are fetched by TMA (documents: one box per 64 dimensions; pages: one per page piece).
// A tile that holds sinks or ends the sequence is gathered row by row (cp.async with zero fill; of
// documents the whole groups of 8 window rows by TMA), so the sinks share the tile of the window's end,
// and rows of no token, NaN in them included, never meet a zero weight. Gathering every tile that way cost 5.2 us a tile against the 1.4 us of its
// products (3 warps issue 256 copies of 512 bytes and their addresses).
//
// CTA = 12 warps, one per SM, each with an equal share of all key tiles (gather_plan.cu):
//   warps 0-7   softmax, a warpgroup per sub-tile, thread = row = TMEM lane: the 128 scores in
//               registers, hidden ones set to -inf from a bit mask per 32 columns, P (bf16) to TMEM, O
//               rescaled there only when the maximum grew by more than 2^8
//   warp 8      MMA issuer and TMEM owner: S_r = Q_r K^T, O_r += P_r V, software-pipelined over the
//               two sub-tiles (P V of the tile before, then S of this one). A whole warp with an elected
//               lane for the MMAs, its index and branches uniform to the compiler, so that the MMAs'
//               operands stay in uniform registers (under `if (lane == 0)`: 260 us instead of 205 for 4 x
//               8192 tokens, 12 heads of 64, window 1024, 16 sinks; 324 instead of 306 for 2 x 8192, 32 / 8
//               heads of 128)
//   warps 9-11  loaders: plain key tiles by TMA (K: warp 9, V: warp 10, a lane per box), Q too where
//               `pack` divides 128; gathered tiles and other Q by 16-byte cp.async into the same
//               128-byte-swizzled layout, its completion signalled by the copies themselves
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

// Bytes that the barrier's current phase awaits, without an arrival.
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// Register split: the softmax rows need all they can get (a spill in their loop goes to L2, the shared
// memory leaves no L1 to speak of, and cost 1.6 times the time); 8 x 216 + 4 x 72 warps' shares use up
// the launch's 12 x 168.
constexpr int kRegsSoftmax = 216;
constexpr int kRegsOther = 72;
static_assert(8 * kRegsSoftmax + 4 * kRegsOther <= 12 * 168, "register split");

// A segment: the key tiles [tb, te) of one row tile and head chunk, and what each sub-tile uses of
// them.
struct GItem {
    int q0, n_tok, behind, chunk, pos0, where, tb, te;
    bool whole;          // all key tiles of the item: rows are written as they are
    bool begins;         // its first key tile is among them
    GatherCols cols;
    int ns;              // columns below it are sinks that lie in the window part
    int unseen;          // pages: columns [ns, unseen) lie below every window and are no sinks: there to begin at
                         // a box
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

__device__ __forceinline__ GatherCols item_cols(const GatherProblem& p, int4 tile, bool paged) {
    return gather_cols(p, tile.z, tile.y & 0xFFFF, gather_align(paged, p.box_rows));
}

__device__ __forceinline__ int key_tiles(const GatherCols& c) { return (c.total + kBlockN - 1) / kBlockN; }

// Walks this CTA's share, segment by segment; the next row tile's words are in flight.
struct GWalk {
    const int4* tiles;
    int x, chunk, tb;        // where the current segment begins
    int ex, echunk, etb;     // where the share ends
    int chunks, n_tiles;
    int4 cur, nxt;
    __device__ __forceinline__ int4 fetch(int i) const {
        return i < n_tiles ? __ldg(tiles + i) : make_int4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void start(const GatherProblem& p, int n) {
        const int4 a = __ldg(p.starts + blockIdx.x), e = __ldg(p.starts + blockIdx.x + 1);
        tiles = p.tiles;
        n_tiles = n;
        chunks = p.heads / p.pack;
        x = a.x;
        chunk = a.y;
        tb = a.z;
        ex = e.x;
        echunk = e.y;
        etb = e.z;
        cur = fetch(x);
        nxt = fetch(x + 1);
    }
    __device__ __forceinline__ bool done() const {
        return x > ex || (x == ex && (chunk > echunk || (chunk == echunk && tb >= etb)));
    }
    __device__ __forceinline__ bool at_end() const { return x == ex && chunk == echunk; }
    __device__ __forceinline__ void advance() {
        tb = 0;
        if (++chunk == chunks) {
            chunk = 0;
            ++x;
            cur = nxt;
            nxt = fetch(x + 1);
        }
    }
};

__device__ __forceinline__ GItem decode_gather(const GWalk& wk, const GatherProblem& p, int p_inv, bool paged) {
    GItem it;
    it.q0 = wk.cur.x;
    it.chunk = wk.chunk;
    it.n_tok = wk.cur.y & 0xFFFF;
    it.behind = wk.cur.y >> 16;
    it.pos0 = wk.cur.z;
    it.where = wk.cur.w;
    it.cols = item_cols(p, wk.cur, paged);
    const int all = key_tiles(it.cols);
    it.tb = wk.tb;
    it.te = wk.at_end() ? wk.etb : all;
    it.begins = it.tb == 0;
    it.whole = it.begins && it.te == all;
    it.ns = p.window > 0 ? p.sinks - it.cols.lo : 0;
    it.unseen = paged && p.window > 0 ? it.pos0 - p.window + 1 - it.cols.lo : 0;
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

// What the MMA issuer and the softmax warps need of a segment, written by loader warp 9 as it reaches
// it, well ahead of them. (Each role decoding for itself put a few hundred instructions, cold in the
// instruction cache, between two items: 4,000 cycles in the MMA warp, 2,200 in the softmax warps.)
struct GBoard {
    int last_one;  // the share is over; nothing else is valid
    int q0, chunk, pos0, tb, te, whole, begins, lo, n_w, total, ns, sf, sl;
    int unseen;
    int nr[2], wf[2], wl[2], first[2], last[2];
    int t_full[2], t_end[2];  // tiles [t_full, t_end) of sub-tile r need no mask
};
constexpr uint32_t kBoards = 4;

struct GBars {
    TcBars t;
    uint64_t stall;  // never signalled: the failure-detection test hook waits on it
    uint64_t item_full[kBoards], item_empty[kBoards];
    GBoard board[kBoards];
};
constexpr int kGBarBytes = 1280;
static_assert(sizeof(GBars) <= kGBarBytes, "barrier block");

template <int HD, bool PAGED>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_gather_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k8,
                       const __grid_constant__ CUtensorMap tm_v8, const GatherProblem p, const int p_inv) {
    using L = TcLayout<HD>;
    constexpr bool kSepP = HD == 64;
    constexpr uint32_t kTmP = kSepP ? L::kTmO + 2 * HD : 0;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw_u32 + 1023u) & ~1023u) - raw_u32);
    const uint32_t sbase = smem_u32(smem);
    static_assert(L::kOffBar + kGBarBytes + 1024 <= 232448, "shared memory budget");
    GBars* gbars = reinterpret_cast<GBars*>(smem + L::kOffBar);
    TcBars* bars = &gbars->t;
    volatile int* abort_flag = &bars->abort;
    int* dev_status = &p.hdr->status;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // (uniform)
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
            for (uint32_t i = 0; i < kBoards; ++i) {
                mbar_init(&gbars->item_full[i], 1);
                mbar_init(&gbars->item_empty[i], 9);  // the MMA warp and 8 softmax warps
            }
            mbar_init(&bars->drain, 1);
            mbar_init(&gbars->stall, 1);
            bars->abort = 0;
            fence_mbar_init();
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
            if (!PAGED) {
                tma_prefetch_desc(&tm_k8);
                tma_prefetch_desc(&tm_v8);
            }
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
    const int n_tiles = *reinterpret_cast<volatile int*>(&p.hdr->n_items);
    const int H = p.heads, G = p.heads / p.kv_heads;

    if (warp >= 8) regs_decrease<kRegsOther>();
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
        const bool q_boxes = kBlockM % p.pack == 0;
        uint32_t qc = 0, kc = 0;  // Q sub-tiles and key tiles issued
        uint32_t k_alone = 0;     // giving up: K of one tile more
        bool ok = true;
        auto acquire = [&](uint64_t* bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, dev_status));
        };
        // address of this lane's unit of row `row` in a swizzled tile
        auto place = [&](uint32_t tile, int row) -> uint32_t {
            return tile + unit_off + row * 128 + (((unit & 7) ^ (row & 7)) << 4);
        };
        // Rows [from, 128) of a K or V tile (`from` a multiple of 8) whose pool rows are i0 .. i3 of lane row % 32
        // for the four blocks of 32 rows (negative: zeros). A small loop: unrolled, this code ran cold every
        // time and took 5,000 cycles a tile.
        auto load_rows = [&](uint32_t tile, const __nv_bfloat16* all, int from, int i0, int i1, int i2, int i3, int head) {
#pragma unroll 2
            for (int j = from / kRpi + w; j < kBlockN / kRpi; j += kLoadWarps) {
                const int row = j * kRpi + row_in;
                const int block = row >> 5;
                const int mine = block == 0 ? i0 : (block == 1 ? i1 : (block == 2 ? i2 : i3));
                const int x = __shfl_sync(0xffffffffu, mine, row & 31);
                const int64_t at = (static_cast<int64_t>(x < 0 ? 0 : x) * p.kv_heads + head) * HD;
                cp_async_16_zfill(place(tile, row), all + at, x < 0 ? 0u : 16u);
            }
        };
        // Documents: rows [0, 8 n) of a gathered tile, window columns all, by TMA in boxes of 8 rows, a lane per
        // box; their bytes are awaited besides the loader threads' arrivals.
        auto load_groups = [&](const CUtensorMap* map, int off, int64_t row0, int n, int head, uint64_t* bar) {
            if (n == 0) return;
            if (lane == 0) mbar_expect_tx(bar, n * 8 * HD * 2);
            __syncwarp();
            if (lane < n) {
#pragma unroll
                for (int c = 0; c < HD / 64; ++c)
                    tma_load_2d(smem + off + c * L::kChunk + lane * 1024, map, head * HD + 64 * c,
                                static_cast<int>(row0) + 8 * lane, bar);
            }
            __syncwarp();
        };
        // 128 consecutive columns by TMA, a lane per box; a page that is none reads as zeros (a row behind
        // the pool). Every loader thread arrives once per tile: here one of them with the bytes to come.
        auto load_boxes = [&](const CUtensorMap* map, int off, const GItem& it, int col0, int head, uint64_t* bar) {
            if (lane == 0) mbar_arrive_expect_tx(bar, L::kKV);
            else mbar_arrive(bar);
            if (lane * p.box_rows < kBlockN) {
                int64_t row = key_row<PAGED>(p, it.where, it.where, it.cols.lo + col0 + lane * p.box_rows);
                if (PAGED && row < 0) {
                    row = static_cast<int64_t>(p.n_pages) << p.page_shift;
                    if (p.status) atomicMax(p.status, DEV_BAD_PAGE);
                }
#pragma unroll
                for (int c = 0; c < HD / 64; ++c)
                    tma_load_2d(smem + off + c * L::kChunk + lane * p.box_rows * 128, map, head * HD + 64 * c,
                                static_cast<int>(row), bar);
            }
            __syncwarp();
        };
        // query sub-tile r of an item
        auto load_q = [&](const GItem& it, int r) -> bool {
            const uint32_t sq = qc % L::kQSlots;
            uint64_t* bar = &bars->q_full[sq];
            if (!acquire(&bars->q_empty[sq], ((qc / L::kQSlots) & 1) ^ 1)) return false;
            ++qc;
            if (q_boxes) {  // (rows behind the tile's last are other queries': nobody stores theirs)
                if (w != 0 || lane != 0) {
                    mbar_arrive(bar);
                } else {
                    mbar_arrive_expect_tx(bar, L::kQSub);
#pragma unroll
                    for (int c = 0; c < HD / 64; ++c)
                        tma_load_3d(smem + L::kOffQ + sq * L::kQSub + c * L::kChunk, &tm_q, 64 * c, it.chunk * p.pack,
                                    it.q0 + div_pack(kBlockM * r, p_inv), bar);
                }
                __syncwarp();
                return true;
            }
            const uint32_t tile = sbase + L::kOffQ + sq * L::kQSub;
            const int64_t base = (static_cast<int64_t>(it.q0) * H + it.chunk * p.pack) * HD;
#pragma unroll 2
            for (int j = w; j < kBlockM / kRpi; j += kLoadWarps) {
                const int row = j * kRpi + row_in, rr = kBlockM * r + row;
                const int tok = div_pack(rr, p_inv);
                const bool in = row < it.nr[r];
                const int64_t at = in ? base + (static_cast<int64_t>(tok) * H + (rr - tok * p.pack)) * HD : base;
                cp_async_16_zfill(place(tile, row), q_all + at, in ? 16u : 0u);
            }
            cp_async_arrive(bar);
            return true;
        };
        uint32_t ic = 0;  // segments published
        auto publish = [&](const GItem* it) -> bool {
            const uint32_t i = ic % kBoards;
            if (!acquire(&gbars->item_empty[i], ((ic / kBoards) & 1) ^ 1)) return false;
            ++ic;
            if (lane == 0) {
                GBoard& b = gbars->board[i];
                b.last_one = it == nullptr;
                if (it) {
                    b.q0 = it->q0;
                    b.chunk = it->chunk;
                    b.pos0 = it->pos0;
                    b.tb = it->tb;
                    b.te = it->te;
                    b.whole = it->whole;
                    b.begins = it->begins;
                    b.lo = it->cols.lo;
                    b.n_w = it->cols.n_w;
                    b.total = it->cols.total;
                    b.ns = it->ns;
                    b.unseen = it->unseen;
                    b.sf = it->sf;
                    b.sl = it->sl;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int nr = it->nr[r], p_lo = it->pos0 - it->cols.lo;  // column of the first token
                        b.nr[r] = nr;
                        b.wf[r] = it->wf[r];
                        b.wl[r] = it->wl[r];
                        b.first[r] = it->first[r];
                        b.last[r] = it->last[r];
                        b.t_full[r] = p.window > 0 ? (p_lo + div_pack(kBlockM * r + nr - 1, p_inv) - p.window + kBlockN) / kBlockN : 0;
                        b.t_end[r] = (p_lo + div_pack(kBlockM * r, p_inv) + 1) / kBlockN;
                    }
                }
                mbar_arrive(&gbars->item_full[i]);
            }
            __syncwarp();
            return true;
        };
        GWalk wk;
        for (wk.start(p, n_tiles); ok && !wk.done(); wk.advance()) {
            const GItem it = decode_gather(wk, p, p_inv, PAGED);
            const int head = it.chunk * p.pack / G;
            if (w == 0) ok = publish(&it);
            if (ok && it.active(0)) ok = load_q(it, 0);
            for (int t = it.tb; ok && t < it.te; ++t, ++kc) {
                const int col0 = t * kBlockN;
                const uint32_t sk = kc % L::kKStages, sv = kc % L::kVStages;
                // all 128 columns are window columns, or tokens of the sequence behind the last one
                const int past = col0 + kBlockN - it.cols.n_w;
                if (p.box_rows >= 8 && (past <= 0 || (it.cols.total == it.cols.n_w && past <= it.behind))) {
                    ok = acquire(&bars->k_empty[sk], ((kc / L::kKStages) & 1) ^ 1);
                    if (!ok) break;
                    if (w == 0) load_boxes(&tm_k, L::kOffK + sk * L::kKV, it, col0, head, &bars->k_full[sk]);
                    else mbar_arrive(&bars->k_full[sk]);
                    ok = acquire(&bars->v_empty[sv], ((kc / L::kVStages) & 1) ^ 1);
                    if (!ok) {
                        k_alone = 1;
                        break;
                    }
                    if (w == 1) load_boxes(&tm_v, L::kOffV + sv * L::kKV, it, col0, head, &bars->v_full[sv]);
                    else mbar_arrive(&bars->v_full[sv]);
                } else {
                    // documents: whole groups of 8 window columns by TMA, the rest row by row. (Pages: the lookups in
                    // between made it slower, 68 us instead of 63 for 24 sequences of 1 to 300 new tokens, 12 heads
                    // of 64, window 1024; documents of 65,536 tokens, 6 paired heads of 128, window 128: 136 instead of 140; 2 x
                    // 8192, 32 / 8 heads of 128, window 1024: 292 instead of 306.)
                    const int plain = it.cols.n_w - col0 < kBlockN ? it.cols.n_w - col0 : kBlockN;
                    const int groups = !PAGED && plain > 0 ? plain >> 3 : 0;
                    int idx[4];
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const int col = col0 + 32 * kk + lane;
                        idx[kk] = -1;
                        if (col >= col0 + 8 * groups && col < it.cols.total) {
                            const int64_t row = key_row<PAGED>(p, it.where, it.where, col_pos(it.cols, col));
                            if (row < 0 && p.status) atomicMax(p.status, DEV_BAD_PAGE);
                            idx[kk] = static_cast<int>(row);
                        }
                    }
                    ok = acquire(&bars->k_empty[sk], ((kc / L::kKStages) & 1) ^ 1);
                    if (!ok) break;
                    if (!PAGED && w == 0)
                        load_groups(&tm_k8, L::kOffK + sk * L::kKV, it.where + it.cols.lo + col0, groups, head, &bars->k_full[sk]);
                    load_rows(sbase + L::kOffK + sk * L::kKV, k_all, 8 * groups, idx[0], idx[1], idx[2], idx[3], head);
                    cp_async_arrive(&bars->k_full[sk]);
                    ok = acquire(&bars->v_empty[sv], ((kc / L::kVStages) & 1) ^ 1);
                    if (!ok) {
                        k_alone = 1;
                        break;
                    }
                    if (!PAGED && w == 1)
                        load_groups(&tm_v8, L::kOffV + sv * L::kKV, it.where + it.cols.lo + col0, groups, head, &bars->v_full[sv]);
                    load_rows(sbase + L::kOffV + sv * L::kKV, v_all, 8 * groups, idx[0], idx[1], idx[2], idx[3], head);
                    cp_async_arrive(&bars->v_full[sv]);
                }
                // the second sub-tile's Q after the first key tile: its slot is free only when the previous
                // item's epilogue is through, and the first sub-tile can start without it
                if (t == it.tb && it.active(1)) ok = load_q(it, 1);
            }
        }
        if (ok && w == 0) ok = publish(nullptr);
        cp_async_wait_all();
        if (!ok && lane == 0) {
            // Wait for the TMA copies issued last into every buffer, with one limit for all: a barrier whose other
            // loaders gave up before they arrived never completes.
            const uint64_t t0 = globaltimer_ns();
            auto drain = [&](uint64_t* bars_of, uint32_t ring, uint32_t issued) {
                for (uint32_t n = issued > ring ? issued - ring : 0; n < issued; ++n)
                    while (!mbar_test(&bars_of[n % ring], (n / ring) & 1) && globaltimer_ns() - t0 <= kWaitLimitNs) {}
            };
            drain(bars->q_full, L::kQSlots, qc);
            drain(bars->k_full, L::kKStages, kc + k_alone);
            drain(bars->v_full, L::kVStages, kc);
        }
        __syncwarp();
    } else if (warp == 8) {
        // ------------------------------------------------------------ MMA issuer
        constexpr uint32_t idesc_qk = idesc_bf16_f32(kBlockM, kBlockN, 0, 0);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(kBlockM, HD, 0, 1);
        uint32_t s_cnt[2] = {0, 0}, p_cnt[2] = {0, 0};  // S and P V products issued per sub-tile
        bool pv_open[2] = {false, false};  // hd 128: the last P V of r not yet seen complete
        // key tile g - 1 as sub-tile r used it: its S was issued, its P V not yet
        bool pend[2] = {false, false}, pend_first[2] = {false, false}, pend_last[2] = {false, false};
        uint32_t qc = 0;  // Q sub-tiles of the segments before the current one
        uint32_t g = 0;   // index of the current key tile in this CTA's stream
        int z_lo = 0, z_hi = 0;  // pages: rows of V_{g-1} that no query sees
        bool ok = true, more = true;
        for (uint32_t ic = 0; ok && more; ++ic) {
            const uint32_t ib = ic % kBoards;
            ok = __all_sync(0xffffffffu, mbar_wait(&gbars->item_full[ib], (ic / kBoards) & 1, abort_flag, dev_status));
            if (!ok) break;
            const GBoard& bd = gbars->board[ib];
            auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
            more = !uniform(bd.last_one);  // behind the last segment: one more turn, for the last P V
            const int tb = more ? uniform(bd.tb) : 0, te = more ? uniform(bd.te) : (g > 0 ? 1 : 0);
            const int sf = uniform(bd.sf), sl = uniform(bd.sl);
            const int ns = PAGED ? uniform(bd.ns) : 0, unseen = PAGED ? uniform(bd.unseen) : 0;
            int nr[2], wf[2], wl[2], first[2], last[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                nr[r] = uniform(bd.nr[r]);
                wf[r] = uniform(bd.wf[r]);
                wl[r] = uniform(bd.wl[r]);
                first[r] = uniform(bd.first[r]);
                last[r] = uniform(bd.last[r]);
            }
            if (lane == 0) mbar_arrive(&gbars->item_empty[ib]);
            uint32_t q_slot[2], q_par[2], n_act = 0;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                q_slot[r] = (qc + n_act) % L::kQSlots;
                q_par[r] = ((qc + n_act) / L::kQSlots) & 1;
                n_act += more && first[r] <= last[r] ? 1 : 0;
            }
            qc += n_act;
            for (int t = tb; t < te; ++t) {
                if (g > 0) {
                    const uint32_t n = g - 1;
                    ok = __all_sync(0xffffffffu, mbar_wait(&bars->v_full[n % L::kVStages], (n / L::kVStages) & 1, abort_flag, dev_status));
                    if (!ok) break;
                    if (PAGED && z_lo < z_hi) {
                        // Their scores are masked, but their values may be anything, and NaN times a zero weight is
                        // NaN: zeros instead (a row is 128 bytes of each chunk). (Fetching that box row by row, with
                        // zeros for them: 80.2 us, this 78.9, neither 77.9, 24 sequences of 1 to 300 new tokens, 12
                        // heads of 64, window 1024, 16 sinks.)
                        uint8_t* v = smem + L::kOffV + (n % L::kVStages) * L::kKV + z_lo * 128;
#pragma unroll 1
                        for (int x = lane; x < (z_hi - z_lo) * 8; x += 32)
#pragma unroll
                            for (int c = 0; c < HD / 64; ++c)
                                *reinterpret_cast<uint4*>(v + c * L::kChunk + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                        z_hi = 0;
                    }
                    fence_proxy_async_smem();  // rows written by cp.async and above; the MMA reads them next
                }
                const uint32_t sk = g % L::kKStages;
                if (more) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&bars->k_full[sk], (g / L::kKStages) & 1, abort_flag, dev_status));
                    if (!ok) break;
                    fence_proxy_async_smem();
                }
                // O_r += P_r V_{g-1}
                auto product_pv = [&](int r, bool is_first, bool is_last) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&bars->p_full[r], p_cnt[r] & 1, abort_flag, dev_status));
                    if (!ok) return;
                    tc_fence_after();
                    const uint32_t a_p = tmem + (kSepP ? kTmP + 64 * r : 128 * r);
                    const uint64_t v0 = desc_v(sbase + L::kOffV + ((g - 1) % L::kVStages) * L::kKV, 0);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < kBlockN / 16; ++kk)  // 2048 bytes on per 16 keys
                            umma_f16_ts(tmem + L::kTmO + HD * r, a_p + 8 * kk, v0 + kk * (2048 >> 4), idesc_pv,
                                        (!is_first || kk > 0) ? 1u : 0u);
                        umma_commit(&bars->pv_done[r]);
                        if (is_last) umma_commit(&bars->o_ready[r]);
                    }
                    __syncwarp();
                    ++p_cnt[r];
                    pv_open[r] = !kSepP;
                };
                // S_r = Q_r K_g^T
                auto product_s = [&](int r) {
                    if (kSepP) {
                        // hd 64: S_r is free once the softmax has read its last tile
                        if (s_cnt[r] > 0)
                            ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_free[r], (s_cnt[r] - 1) & 1, abort_flag, dev_status));
                    } else if (pv_open[r]) {
                        // hd 128: S_r overwrites the columns that P_r shares with it
                        ok = __all_sync(0xffffffffu, mbar_wait(&bars->pv_done[r], (p_cnt[r] - 1) & 1, abort_flag, dev_status));
                        pv_open[r] = false;
                    }
                    if (ok && t == first[r]) {
                        ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_full[q_slot[r]], q_par[r], abort_flag, dev_status));
                        fence_proxy_async_smem();
                    }
                    if (!ok) return;
                    tc_fence_after();
                    const uint64_t q0 = desc_kmajor(sbase + L::kOffQ + q_slot[r] * L::kQSub, 0);
                    const uint64_t k0 = desc_kmajor(sbase + L::kOffK + sk * L::kKV, 0);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk) {  // (as desc_kmajor steps)
                            const uint32_t step = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                            umma_f16_ss(tmem + 128 * r, q0 + step, k0 + step, idesc_qk, kk == 0 ? 0u : 1u);
                        }
                        umma_commit(&bars->s_full[r]);
                        if (t == last[r]) umma_commit(&bars->q_empty[q_slot[r]]);
                    }
                    __syncwarp();
                    ++s_cnt[r];
                    pend[r] = true;
                    pend_first[r] = t == first[r];
                    pend_last[r] = t == last[r];
                };
                // Sub-tile by sub-tile; hd 64: S, then P V of the tile before; hd 128 (P over S): the other
                // way round. A segment's first S_1 may have to wait for the epilogue of the last one's
                // sub-tile 0 (its Q slot), whose P V comes before it here. One copy of each product:
                // this warp's code is fetched anew whenever the softmax loop has pushed it out.
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const bool uses = more && nr[r] > 0 && ((t >= wf[r] && t <= wl[r]) || (t >= sf && t <= sl));
                    const bool pv = pend[r], pv_first = pend_first[r], pv_last = pend_last[r];
                    pend[r] = false;
                    if (kSepP && ok && uses) product_s(r);
                    if (ok && pv) product_pv(r, pv_first, pv_last);
                    if (!kSepP && ok && uses) product_s(r);
                }
                if (!ok || !more) break;
                if (elect_one()) {
                    if (g > 0) umma_commit(&bars->v_empty[(g - 1) % L::kVStages]);
                    umma_commit(&bars->k_empty[sk]);
                }
                __syncwarp();
                if (PAGED && t == 0) {
                    z_lo = ns > 0 ? ns : 0;
                    z_hi = unseen;
                }
                ++g;
            }
        }
        // Wait (bounded) until every MMA this warp issued has finished.
        if (elect_one()) umma_commit(&bars->drain);
        __syncwarp();
        drain_wait(&bars->drain, 0);
    } else {
        // ------------------------------------------------------------ softmax, sub-tile r
        regs_increase<kRegsSoftmax>();
        const int r = warp >> 2;
        const int row = threadIdx.x & 127;  // row of the sub-tile == TMEM lane
        const int r0 = (warp & 3) * 32;     // first row of this warp
        const uint32_t tm_lane = tmem + (static_cast<uint32_t>(r0) << 16);
        const uint32_t tm_s = tm_lane + 128 * r;
        const uint32_t tm_p = kSepP ? tm_lane + kTmP + 64 * r : tm_s;
        const uint32_t tm_o = tm_lane + L::kTmO + HD * r;
        const float scale_log2 = p.scale * kLog2e;
        const uint64_t scale2 = f32x2(scale_log2, scale_log2);
        uint32_t s_cnt = 0, o_cnt = 0;
        uint32_t pv_seen = 0;  // hd 64: P V completions of this sub-tile awaited so far
        uint32_t q_seq = 0;    // index of the current item's first Q sub-tile in this CTA's stream
        bool ok = true;
        if (p.test_stall_us > 0)  // the wait runs out: status 3, and every role winds down
            ok = __all_sync(0xffffffffu, mbar_wait(&gbars->stall, 0, abort_flag, dev_status,
                                                   1000ull * static_cast<uint64_t>(p.test_stall_us)));
        // the low n bits (n clamped to 0 .. 32)
        auto low_bits = [](int n) -> uint32_t { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); };
        for (uint32_t ic = 0; ok; ++ic) {
            const uint32_t ib = ic % kBoards;
            ok = __all_sync(0xffffffffu, mbar_wait(&gbars->item_full[ib], (ic / kBoards) & 1, abort_flag, dev_status));
            if (!ok) break;
            const GBoard& bd = gbars->board[ib];
            const int last_one = bd.last_one, q0 = bd.q0, chunk = bd.chunk, whole = bd.whole, begins = bd.begins;
            const int first_col = bd.pos0 - bd.lo, b_n_w = bd.n_w, b_total = bd.total, ns = bd.ns, sf = bd.sf;
            const int nr = bd.nr[r], t_first = bd.first[r], t_last = bd.last[r], wl = bd.wl[r];
            const int t_full = bd.t_full[r], t_end = bd.t_end[r];
            const int act0 = bd.first[0] <= bd.last[0], act1 = bd.first[1] <= bd.last[1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&gbars->item_empty[ib]);
            if (last_one) break;
            const uint32_t my_q = q_seq + (r ? act0 : 0);
            q_seq += act0 + act1;
            if (nr == 0) continue;
            const bool valid = row < nr;
            const int tok = div_pack(kBlockM * r + row, p_inv);
            // a cut item's rows: place 2 c of CTA c for a segment that continues an item (its first), 2 c
            // + 1 for one that begins it (its last)
            const int part_row = (2 * static_cast<int>(blockIdx.x) + begins) * kGatherRows + kBlockM * r + row;
            if (t_first > t_last) {  // no columns of this segment: an empty partial row
                if (valid) p.part_lse[part_row] = -INFINITY;
                continue;
            }
            // this row's visible columns: (c_hi - window, c_hi] and those below ns, of the window part,
            // and the sink columns [n_w, total)
            const int c_hi = valid ? first_col + tok : -1;
            const int n_w = valid ? b_n_w : 0, total = valid ? b_total : 0;
            float m = -INFINITY, l = 0.f;
            // window tiles up to wl, then the sinks'
            for (int t = t_first; t <= t_last; t = (t >= wl && t + 1 < sf) ? sf : t + 1) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full[r], s_cnt & 1, abort_flag, dev_status));
                if (!ok) break;
                ++s_cnt;
                tc_fence_after();
                uint64_t sum_a = f32x2(0.f, 0.f), sum_b = f32x2(0.f, 0.f);
                float mx = -INFINITY, alpha = 1.0f;
                uint64_t negm2 = 0;
                bool rescale = false;
                // After the scores' maximum is known: the reference stays until the maximum has grown by more
                // than 2^8 (O / l and the lse are exact for any reference).
                auto new_reference = [&]() {
                    const float m_new = fmaxf(m, mx * scale_log2);
                    rescale = m_new > m + 8.0f;
                    alpha = rescale ? ex2(m - m_new) : 1.0f;
                    if (rescale) m = m_new;
                    const float neg_m = (m == -INFINITY) ? 0.f : -m;
                    negm2 = f32x2(neg_m, neg_m);
                };
                // hd 64: the last P V reads P_r and adds into O_r; it must be complete before P_r is overwritten
                // and O_r rescaled
                auto wait_pv = [&]() {
                    if (kSepP && pv_seen < s_cnt - 1) {
                        ok = __all_sync(0xffffffffu, mbar_wait(&bars->pv_done[r], pv_seen & 1, abort_flag, dev_status));
                        ++pv_seen;
                        tc_fence_after();
                    }
                };
                const bool masked = t < t_full || t >= t_end;
                auto visible = [&](int c) -> uint32_t {  // bit e: column 32 c + e of the tile is visible
                    const int cb = t * kBlockN + 32 * c;
                    const uint32_t below = p.window > 0 ? low_bits(c_hi + 1 - p.window - cb) : 0u;
                    const uint32_t seen = low_bits(c_hi + 1 - cb) & (~below | low_bits(ns - cb));
                    return seen | (low_bits(total - cb) & ~low_bits(n_w - cb));
                };
                // the 128 scores at once, in registers
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
                if (masked) {
                    uint32_t vis[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) vis[c] = visible(c);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            v[32 * c + e] = ((vis[c] >> e) & 1u) ? v[32 * c + e] : __float_as_uint(-INFINITY);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) mx = fmaxf(mx, chunk_max<kMaskNone>(v + 32 * c, 0, 0, 0));
                new_reference();
                // P = 2^(s scale log2 e - m), written after the whole row was read (it may share S's columns)
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    chunk_exp<kMaskNone>(v + 32 * c, 0, 0, 0, scale2, negm2, sum_a, sum_b, pk + 16 * (c & 1));
                    if (c == 1) wait_pv();
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
#pragma unroll 1  // (rare: small code before speed)
                    for (int c = 0; c < HD / 32; ++c) {
                        uint32_t ov[32];
                        tmem_ld32(tm_o + 32 * c, ov);
                        tmem_wait_ld();
                        regs_after_wait(ov);
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                        tmem_st32(tm_o + 32 * c, ov);
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
            // O a chunk of 32 columns at a time, in loops: what the softmax warps run has to stay small
            // (unrolled epilogues for both cases below cost 1.3 times the kernel's time in instruction
            // fetches)
            if (!whole) {
                // a partial row: normalised o in float32 and log2 of its sum of exponentials
                float* dst = p.part_o + static_cast<int64_t>(part_row) * HD;
#pragma unroll 1
                for (int c = 0; c < HD / 32; ++c) {
                    uint32_t ov[32];
                    tmem_ld32(tm_o + 32 * c, ov);
                    tmem_wait_ld();
                    regs_after_wait(ov);
                    if (valid)
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(dst + 32 * c + e) =
                                make_float4(__uint_as_float(ov[e]) * inv_l, __uint_as_float(ov[e + 1]) * inv_l,
                                            __uint_as_float(ov[e + 2]) * inv_l, __uint_as_float(ov[e + 3]) * inv_l);
                }
                if (valid) p.part_lse[part_row] = l != 0.f ? m + log2f(l) : -INFINITY;  // (NaN stays)
            } else {
                const int out_row = tok * H + chunk * p.pack + (kBlockM * r + row - tok * p.pack);  // from q0's
                // O -> bf16 through this sub-tile's Q slot (its last S has completed): each warp stages
                // its 32 rows (16-byte units swizzled) and copies them out whole rows at a time; the
                // rows of a token's packed heads lie next to one another in memory
                constexpr int kUnitsO = HD / 8;
                uint8_t* stage = smem + L::kOffQ + (my_q % L::kQSlots) * L::kQSub + (warp & 3) * 32 * (HD * 2);
#pragma unroll 1
                for (int c = 0; c < HD / 32; ++c) {
                    uint32_t ov[32];
                    tmem_ld32(tm_o + 32 * c, ov);
                    tmem_wait_ld();
                    regs_after_wait(ov);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t* w8 = ov + 8 * e;
                        const int u = 4 * c + e;
                        *reinterpret_cast<uint4*>(stage + lane * (HD * 2) + ((u ^ (lane & (kUnitsO - 1))) << 4)) = make_uint4(
                            pack_bf16x2(__uint_as_float(w8[0]) * inv_l, __uint_as_float(w8[1]) * inv_l),
                            pack_bf16x2(__uint_as_float(w8[2]) * inv_l, __uint_as_float(w8[3]) * inv_l),
                            pack_bf16x2(__uint_as_float(w8[4]) * inv_l, __uint_as_float(w8[5]) * inv_l),
                            pack_bf16x2(__uint_as_float(w8[6]) * inv_l, __uint_as_float(w8[7]) * inv_l));
                    }
                }
                __syncwarp();
                constexpr int kRowsPerIter = 32 / kUnitsO;
#pragma unroll 4
                for (int j = 0; j < kUnitsO; ++j) {
                    const int rl = j * kRowsPerIter + lane / kUnitsO, u = lane % kUnitsO;
                    const int ro = __shfl_sync(0xffffffffu, out_row, rl);
                    if (r0 + rl < nr) {
                        const uint4 w4 = *reinterpret_cast<const uint4*>(stage + rl * (HD * 2) + ((u ^ (rl & (kUnitsO - 1))) << 4));
                        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) +
                                             (static_cast<int64_t>(q0) * H + ro) * HD + u * 8;
                        *reinterpret_cast<uint4*>(dst) = w4;
                    }
                }
                if (valid && p.lse) p.lse[static_cast<int64_t>(q0) * H + out_row] = (m + log2f(l)) * kLn2;
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

// Whether boundary a lies at or before boundary (x, chunk, key tile).
__device__ __forceinline__ bool at_or_before(int4 a, int x, int chunk, int t) {
    return a.x < x || (a.x == x && (a.y < chunk || (a.y == chunk && a.z <= t)));
}

// Block (c, 32-row group): where CTA c's share ends inside an item that it began, the item's rows from
// its parts: o = sum 2^(lse_i - max) o_i / sum 2^(lse_i - max), in order. Warp = row.
template <int HD>
__global__ void __launch_bounds__(256) attn_join_cuts_kernel(GatherProblem p, int p_inv) {
    grid_dep_wait();
    if (p.hdr->status == DEV_TIMEOUT) return;  // parts may be missing
    const int c = blockIdx.x, lane = threadIdx.x & 31;
    const int4 cut = p.starts[c + 1];
    if (cut.z == 0 || !at_or_before(p.starts[c], cut.x, cut.y, 0)) return;
    const int4 tile = p.tiles[cut.x];
    const int n_rows = (tile.y & 0xFFFF) * p.pack;
    // parts: this CTA's place 2 c + 1, then place 2 i of the CTAs up to the one that ends the item
    int end = c + 1;
    while (end + 1 < p.n_cta && p.starts[end + 1].x == cut.x && p.starts[end + 1].y == cut.y) ++end;
    for (int k = 0; k < 4; ++k) {
        const int rr = blockIdx.y * 32 + k * 8 + (threadIdx.x >> 5);
        if (rr >= n_rows) return;
        const int tok = div_pack(rr, p_inv);
        const int64_t row = (static_cast<int64_t>(tile.x) + tok) * p.heads + cut.y * p.pack + (rr - tok * p.pack);
        float acc[HD / 32], sum = 0.f, top = -INFINITY;
#pragma unroll
        for (int e = 0; e < HD / 32; ++e) acc[e] = 0.f;
        for (int i = c; i <= end; ++i) {
            // (a share without steps has left nothing)
            const int4 a = p.starts[i], z = p.starts[i + 1];
            if (i > c && a.x == z.x && a.y == z.y && a.z == z.z) continue;
            const int64_t part = (2 * static_cast<int64_t>(i) + (i == c ? 1 : 0)) * kGatherRows + rr;
            const float lse = p.part_lse[part];
            if (lse == -INFINITY) continue;  // an empty part (its o is not written)
            const float m = fmaxf(top, lse), old = exp2f(top - m), w = exp2f(lse - m);
            top = m;
            sum = sum * old + w;
#pragma unroll
            for (int e = 0; e < HD / 32; ++e) acc[e] = fmaf(w, p.part_o[part * HD + 32 * e + lane], acc[e] * old);
        }
        const float inv = 1.f / sum;
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + row * HD;
#pragma unroll
        for (int e = 0; e < HD / 32; ++e) o[32 * e + lane] = __float2bfloat16_rn(acc[e] * inv);
        if (p.lse && lane == 0) p.lse[row] = (top + log2f(sum)) * kLn2;
    }
}

template <int HD, bool PAGED>
cudaError_t launch_gather_hd(const GatherProblem& p, const CUtensorMap& tq, const CUtensorMap& tk,
                             const CUtensorMap& tv, const CUtensorMap& tk8, const CUtensorMap& tv8,
                             cudaStream_t stream) {
    constexpr int kSmem = TcLayout<HD>::kOffBar + kGBarBytes + 1024;  // + slack to align to 1024
    cudaError_t e = cudaFuncSetAttribute(attn_gather_kernel<HD, PAGED>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const int p_inv = (65536 + p.pack - 1) / p.pack;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.n_cta);
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attn_gather_kernel<HD, PAGED>, tq, tk, tv, tk8, tv8, p, p_inv);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(p.n_cta, (p.tile_tokens * p.pack + 31) / 32);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attn_join_cuts_kernel<HD>, p, p_inv);
}

}  // namespace

cudaError_t launch_attn_gather(const GatherProblem& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                               const CUtensorMap& tm_v, const CUtensorMap& tm_k8, const CUtensorMap& tm_v8,
                               cudaStream_t stream) {
    if (p.head_dim != 64 && p.head_dim != 128) return cudaErrorInvalidValue;
    const bool paged = p.kv_lens != nullptr;
    auto* const launch = p.head_dim == 128 ? (paged ? launch_gather_hd<128, true> : launch_gather_hd<128, false>)
                                           : (paged ? launch_gather_hd<64, true> : launch_gather_hd<64, false>);
    return launch(p, tm_q, tm_k, tm_v, tm_k8, tm_v8, stream);
}

}  // namespace pha
