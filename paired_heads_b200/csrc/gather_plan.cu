// gather_plan.cu -- lays out the work of the gathering attention kernel from the lengths on the device:
// the row tiles of all sequences, and equal shares of their key tiles for the CTAs.
//
// One CTA: lengths checked and row tiles counted per sequence, a scan over the sequences, a scan over
// the row tiles of their steps (key tiles, one more for an item's fixed costs, times the head chunks),
// and a binary search for the start of each share. Equal shares of the steps keep every SM busy to the
// end whatever the lengths: handing out whole items left SMs idle in the last round (256 equal items
// on 148 SMs: 0.86 of the time used). It takes 7 us for 133 documents of 65,536 tokens: scans and searches
// that wait for one another.
#include <cuda_runtime.h>
#include <stdint.h>

#include "gather.cuh"
#include "scan.cuh"

namespace pha {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanNear = 2048;        // sequences whose tile counts are kept in shared memory
constexpr int kPlanNearSteps = 3000;   // row tiles whose steps are

__global__ void __launch_bounds__(kPlanThreads) gather_plan_kernel(GatherProblem p, int64_t max_tiles,
                                                                   int* __restrict__ before_far,
                                                                   int64_t* __restrict__ steps_far, int strict) {
    __shared__ int64_t near_steps[kPlanNearSteps + 1];
    __shared__ int64_t sums[kPlanThreads / 32];
    __shared__ int near[kPlanNear];
    __shared__ int bad;
    grid_dep_launch();  // the attention kernel's prologue may start
    const int tid = threadIdx.x;
    int* before = p.batch <= kPlanNear ? near : before_far;
    if (tid == 0) bad = 0;
    __syncthreads();
    // row tiles per sequence, and their places
    int64_t n_tiles = 0;
    for (int base = 0; base < p.batch; base += kPlanThreads) {
        const int b = base + tid;
        int64_t n = 0;
        if (b < p.batch) {
            const GatherSeq s = gather_seq(p, b);
            if (!s.ok) atomicOr(&bad, 1);
            n = max_tiles > 0 ? (s.n_q + p.tile_tokens - 1) / p.tile_tokens : 0;
        }
        int64_t chunk;
        const int64_t ex = cta_exclusive_scan<kPlanThreads>(n, sums, chunk);
        if (b < p.batch) before[b] = static_cast<int>(n_tiles + ex);
        n_tiles += chunk;
    }
    __syncthreads();
    const int code = bad && strict ? DEV_BAD_SEQLENS : (n_tiles > max_tiles ? DEV_OVERFLOW : DEV_OK);
    if (tid == 0) {
        const int report = bad ? DEV_BAD_SEQLENS : code;  // (overlapping sequences, too many tiles: bad lengths first)
        p.hdr->n_items = code == DEV_OK ? static_cast<int>(n_tiles) : 0;
        p.hdr->status = report;
        if (p.status && report != DEV_OK) atomicMax(p.status, report);
    }
    if (max_tiles == 0) return;
    const int chunks = p.heads / p.pack;
    int64_t* steps = n_tiles <= kPlanNearSteps ? near_steps : steps_far;
    int64_t total = 0;
    if (code == DEV_OK) {
        for (int64_t base = 0; base < n_tiles; base += kPlanThreads) {
            const int64_t x = base + tid;
            int64_t cost = 0;
            if (x < n_tiles) {
                int b = 0, hi = p.batch;  // last sequence with before[b] <= x (skips those without tiles)
                while (hi - b > 1) {
                    const int mid = (b + hi) >> 1;
                    if (before[mid] <= x) b = mid; else hi = mid;
                }
                const GatherSeq s = gather_seq(p, b);
                const int t0 = static_cast<int>(x - before[b]) * p.tile_tokens;
                const int n = s.n_q - t0 < p.tile_tokens ? s.n_q - t0 : p.tile_tokens;
                const int pos0 = s.kv - s.n_q + t0;
                const int behind = s.kv - pos0 - n < 127 ? s.kv - pos0 - n : 127;
                p.tiles[x] = make_int4(static_cast<int>(s.q0) + t0, n | (behind << 16), pos0,
                                       p.kv_lens ? b : static_cast<int>(s.base));
                const GatherCols c = gather_cols(p, pos0, n, gather_align(p.kv_lens != nullptr, p.box_rows));
                cost = static_cast<int64_t>((c.total + kBlockN - 1) / kBlockN + 1) * chunks;
            }
            int64_t chunk;
            const int64_t ex = cta_exclusive_scan<kPlanThreads>(cost, sums, chunk);
            if (x < n_tiles) steps[x] = total + ex;
            total += chunk;
        }
        if (tid == 0) steps[n_tiles] = total;
    }
    __syncthreads();
    // shares of at least kGatherMinSteps steps
    const int64_t most = (total + kGatherMinSteps - 1) / kGatherMinSteps;
    const int64_t n_cta = most < p.n_cta ? (most > 0 ? most : 1) : p.n_cta;
    for (int c = tid; c <= p.n_cta; c += kPlanThreads) {
        int4 start = make_int4(static_cast<int>(code == DEV_OK ? n_tiles : 0), 0, 0, 0);  // the end
        const int64_t at = c < n_cta ? total * c / n_cta : total;
        if (at < total) {
            int64_t x = 0, hi = n_tiles;
            while (hi - x > 1) {
                const int64_t mid = (x + hi) >> 1;
                if (steps[mid] <= at) x = mid; else hi = mid;
            }
            const int64_t each = (steps[x + 1] - steps[x]) / chunks, in = at - steps[x];
            const int64_t s = in % each;  // step 0 is the fixed cost
            start = make_int4(static_cast<int>(x), static_cast<int>(in / each), static_cast<int>(s > 0 ? s - 1 : 0), 0);
        }
        p.starts[c] = start;
    }
}

}  // namespace

cudaError_t launch_gather_plan(const GatherProblem& p, int64_t max_tiles, int* before, int64_t* steps,
                               bool strict, cudaStream_t stream) {
    gather_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p, max_tiles, before, steps, strict ? 1 : 0);
    return cudaGetLastError();
}

}  // namespace pha
