// gather_plan.cu -- work list of the gathering attention kernel: (sequence, token tile, head chunk,
// split of the key tiles) items from the lengths on the device, most key tiles first.
//
// One CTA: lengths checked and tiles counted per sequence, a scan over the sequences, a histogram of
// the tiles' costs (their key tiles), a scan of it from the costliest down, and emission, one thread a
// tile. Items of equal cost may come out in any order; results do not depend on it.
#include <cuda_runtime.h>
#include <stdint.h>

#include "gather.cuh"
#include "scan.cuh"

namespace pha {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanBuckets = 4096;  // costs from the last one up share it

struct PlanTile {
    int64_t q0;           // first q slot
    int n, pos0;          // tokens, position of the first
    int tiles;            // key tiles
    int where;            // item word w0
};

__device__ __forceinline__ PlanTile plan_tile(const GatherProblem& p, int b, int t) {
    const GatherSeq s = gather_seq(p, b);
    PlanTile x;
    const int t0 = t * p.tile_tokens;
    x.q0 = s.q0 + t0;
    x.n = s.n_q - t0 < p.tile_tokens ? s.n_q - t0 : p.tile_tokens;
    x.pos0 = s.kv - s.n_q + t0;
    x.tiles = (gather_cols(p, x.pos0, x.n).total + kBlockN - 1) / kBlockN;
    x.where = p.kv_lens ? b : static_cast<int>(s.base);
    return x;
}

__global__ void __launch_bounds__(kPlanThreads) gather_plan_kernel(GatherProblem p, int64_t capacity,
                                                                   int* __restrict__ before, int strict) {
    __shared__ int hist[kPlanBuckets];
    __shared__ int sums[kPlanThreads / 32];
    __shared__ int bad;
    grid_dep_launch();  // the attention kernel's prologue may start
    const int tid = threadIdx.x;
    for (int c = tid; c < kPlanBuckets; c += kPlanThreads) hist[c] = 0;
    if (tid == 0) bad = 0;
    __syncthreads();
    // tiles per sequence, and their places
    int n_tiles = 0;
    for (int base = 0; base < p.batch; base += kPlanThreads) {
        const int b = base + tid;
        int n = 0;
        if (b < p.batch) {
            const GatherSeq s = gather_seq(p, b);
            if (!s.ok) atomicOr(&bad, 1);
            n = (s.n_q + p.tile_tokens - 1) / p.tile_tokens;
        }
        int chunk;
        const int ex = cta_exclusive_scan<kPlanThreads>(n, sums, chunk);
        if (b < p.batch) before[b] = n_tiles + ex;
        n_tiles += chunk;
    }
    __syncthreads();
    const int chunks = p.heads / p.pack;
    const int64_t n_items = static_cast<int64_t>(n_tiles) * chunks * p.n_splits;
    const int code = bad && strict ? DEV_BAD_SEQLENS : (n_items > capacity ? DEV_OVERFLOW : DEV_OK);
    if (tid == 0) {
        const int report = code != DEV_OK ? code : (bad ? DEV_BAD_SEQLENS : DEV_OK);
        p.hdr->n_items = code == DEV_OK ? static_cast<int>(n_items) : 0;
        p.hdr->status = report;
        if (p.status && report != DEV_OK) atomicMax(p.status, report);
    }
    if (code != DEV_OK || !p.items) return;  // (without a list: the lengths were only checked)

    auto seq_of = [&](int x) {  // last b with before[b] <= x (skips sequences without tiles)
        int lo = 0, hi = p.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before[mid] <= x) lo = mid; else hi = mid;
        }
        return lo;
    };
    auto bucket = [](int tiles) { return tiles < kPlanBuckets ? tiles : kPlanBuckets - 1; };
    for (int x = tid; x < n_tiles; x += kPlanThreads) {
        const int b = seq_of(x);
        atomicAdd(&hist[bucket(plan_tile(p, b, x - before[b]).tiles)], 1);
    }
    __syncthreads();
    int carry = 0;
    for (int base = 0; base < kPlanBuckets; base += kPlanThreads) {  // from the costliest down
        const int c = kPlanBuckets - 1 - (base + tid);
        int total;
        const int ex = cta_exclusive_scan<kPlanThreads>(hist[c], sums, total);
        hist[c] = carry + ex;
        carry += total;
    }
    __syncthreads();
    for (int x = tid; x < n_tiles; x += kPlanThreads) {
        const int b = seq_of(x);
        const PlanTile t = plan_tile(p, b, x - before[b]);
        int64_t at = static_cast<int64_t>(atomicAdd(&hist[bucket(t.tiles)], 1)) * chunks * p.n_splits;
        for (int h = 0; h < chunks; ++h)
            for (int s = 0; s < p.n_splits; ++s, ++at) {
                p.items[2 * at] = make_int4(static_cast<int>(t.q0), (h << 16) | t.n, t.pos0, t.where);
                p.items[2 * at + 1] = make_int4(
                    static_cast<int>(static_cast<int64_t>(t.tiles) * s / p.n_splits),
                    static_cast<int>(static_cast<int64_t>(t.tiles) * (s + 1) / p.n_splits), s, 0);
            }
    }
}

}  // namespace

cudaError_t launch_gather_plan(const GatherProblem& p, int64_t capacity, int* before, bool strict,
                               cudaStream_t stream) {
    gather_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p, capacity, before, strict ? 1 : 0);
    return cudaGetLastError();
}

}  // namespace pha
