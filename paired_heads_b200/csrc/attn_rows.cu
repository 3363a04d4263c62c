// attn_rows.cu -- attention with window, sinks and pages on CUDA cores (float32 inputs), and the
// join of split key ranges.
//
// One warp per (q slot, head, split of the key columns). A step takes 32 columns: lane = column for
// the scores (its key row read 16 bytes at a time against the query in shared memory), then lane =
// dimension for o += w v (each value row read by the whole warp, coalesced), with the running
// maximum and sum of the softmax between them. All sums are float32. What bounds it is the issue of
// loads and of the multiply-adds, and rows share no reads: the float32 path serves exactness, not
// throughput (5.8 us for documents of 64, 1, 37 and 130 tokens with 4 heads of 16; 373 us, 2.6 TFLOP/s, for
// 8 x 512 tokens, 8 heads of 64, window 128; 3.2 ms, 1.3 TB/s, for 64 single tokens over 8,192, 32 / 8 heads of
// 128; the join takes 5.4 us for 32 sequences of 6 heads of 128 and
// 3 ranges, beside the time of its launch).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gather.cuh"

namespace pha {

namespace {

constexpr int kRowWarps = 4;
constexpr int kMaxDim = 128;
constexpr float kRowsLog2e = 1.4426950408889634f;
constexpr float kRowsLn2 = 0.6931471805599453f;

__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <bool PAGED>
__global__ void __launch_bounds__(32 * kRowWarps) attn_rows_kernel(GatherProblem p) {
    __shared__ __align__(16) float qs[kRowWarps][kMaxDim];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t rows = static_cast<int64_t>(p.total_q) * p.mult * p.heads;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowWarps + warp;
    // the lengths of every sequence, those without a row of q too (documents: the plan has checked them)
    if (PAGED && p.status && blockIdx.x == 0 && blockIdx.y == 0)
        for (int b = threadIdx.x; b < p.batch; b += 32 * kRowWarps)
            if (!gather_seq(p, b).ok) atomicMax(p.status, DEV_BAD_SEQLENS);
    if (row >= rows || (p.hdr && p.hdr->status != DEV_OK)) return;
    const int64_t slot = row / p.heads;
    const int h = static_cast<int>(row % p.heads), g = h / (p.heads / p.kv_heads);
    const int D = p.head_dim, split = blockIdx.y;
    const int b = gather_seq_of(p.cu, p.batch, static_cast<int>(slot / p.mult));
    if (b < 0) return;
    const GatherSeq s = gather_seq(p, b);
    if (!s.ok || slot >= s.q0 + s.n_q) return;  // (behind the last sequence)
    // the columns of the whole sequence's queries when ranges are split (every split is of those)
    const int pos = s.kv - s.n_q + static_cast<int>(slot - s.q0);
    const GatherCols cols = gather_cols(p, pos, 1);
    const GatherCols all = p.split_keys > 0 ? gather_cols(p, s.kv - s.n_q, s.n_q) : cols;
    const bool alone = p.split_keys <= 0 || all.total <= p.split_keys;
    int c0 = 0, c1 = cols.total;
    if (p.split_keys > 0) {
        // splits are counted over this row's own columns; their number bounds the sequence's
        c0 = split * p.split_keys;
        c1 = c0 + p.split_keys < cols.total ? c0 + p.split_keys : cols.total;
        if (c0 >= all.total) return;
    }
    const float* q = static_cast<const float*>(p.q) + row * D;
    for (int d = lane; d < D; d += 32) qs[warp][d] = q[d];
    __syncwarp();
    const float scale2 = p.scale * kRowsLog2e;
    const int64_t stride = static_cast<int64_t>(p.kv_heads) * D;
    const float* kb = static_cast<const float*>(p.k) + static_cast<int64_t>(g) * D;
    const float* vb = static_cast<const float*>(p.v) + static_cast<int64_t>(g) * D;
    float acc[kMaxDim / 32] = {0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    for (int c = c0; c < c1; c += 32) {
        const int col = c + lane;
        int64_t kr = 0;
        float x = -INFINITY;
        if (col < c1) {
            kr = key_row<PAGED>(p, b, s.base, col_pos(cols, col));
            if (kr < 0) {
                if (p.status) atomicMax(p.status, DEV_BAD_PAGE);
                kr = 0;
            }
            const float* k = kb + kr * stride;
            float dot = 0.f;
            if (D % 4 == 0) {  // rows are 16-byte aligned
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                for (int d = 0; d < D; d += 4) {
                    const float4 k4 = __ldg(reinterpret_cast<const float4*>(k + d));
                    const float4 q4 = *reinterpret_cast<const float4*>(&qs[warp][d]);
                    part[0] = fmaf(q4.x, k4.x, part[0]);
                    part[1] = fmaf(q4.y, k4.y, part[1]);
                    part[2] = fmaf(q4.z, k4.z, part[2]);
                    part[3] = fmaf(q4.w, k4.w, part[3]);
                }
                dot = (part[0] + part[1]) + (part[2] + part[3]);
            } else {
                for (int d = 0; d < D; ++d) dot = fmaf(qs[warp][d], k[d], dot);
            }
            x = dot * scale2;
        }
        float mx = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float m_new = fmaxf(m, mx);
        const float alpha = m_new > m ? exp2f(m - m_new) : 1.f;
        const float w = col < c1 ? exp2f(x - m_new) : 0.f;
        float sum = w;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = l * alpha + sum;
        m = m_new;
#pragma unroll
        for (int t = 0; t < kMaxDim / 32; ++t) acc[t] *= alpha;
        const int n = c1 - c < 32 ? c1 - c : 32;
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            const float* v = vb + __shfl_sync(0xffffffffu, kr, j) * stride;
#pragma unroll
            for (int t = 0; t < kMaxDim / 32; ++t)
                if (lane + 32 * t < D) acc[t] = fmaf(wj, v[lane + 32 * t], acc[t]);
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    if (alone) {
        float* o = static_cast<float*>(p.o) + row * D;
#pragma unroll
        for (int t = 0; t < kMaxDim / 32; ++t)
            if (lane + 32 * t < D) o[lane + 32 * t] = acc[t] * inv;
        if (p.lse && lane == 0) p.lse[row] = (m + log2f(l)) * kRowsLn2;
    } else {
        float* o = p.part_o + (split * rows + row) * D;
#pragma unroll
        for (int t = 0; t < kMaxDim / 32; ++t)
            if (lane + 32 * t < D) o[lane + 32 * t] = acc[t] * inv;
        if (lane == 0) p.part_lse[split * rows + row] = l != 0.f ? m + log2f(l) : -INFINITY;  // (NaN stays)
    }
}

// Warp per row: o = sum_s 2^(lse_s - max) o_s / sum_s 2^(lse_s - max) over the row's splits.
template <typename T>
__global__ void __launch_bounds__(32 * kRowWarps) attn_join_kernel(GatherProblem p) {
    grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t rows = static_cast<int64_t>(p.total_q) * p.mult * p.heads;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int64_t slot = row / p.heads;
    const int b = gather_seq_of(p.cu, p.batch, static_cast<int>(slot / p.mult));
    if (b < 0) return;
    const GatherSeq s = gather_seq(p, b);
    if (!s.ok || slot >= s.q0 + s.n_q) return;
    const GatherCols all = gather_cols(p, s.kv - s.n_q, s.n_q);
    const int n = (all.total + p.split_keys - 1) / p.split_keys;
    if (n <= 1) return;  // written by its only split
    float top = -INFINITY;
    for (int i = 0; i < n; ++i) top = fmaxf(top, p.part_lse[i * rows + row]);
    float acc[kMaxDim / 32] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
    for (int i = 0; i < n; ++i) {
        const float part = p.part_lse[i * rows + row];
        if (part == -INFINITY) continue;  // an empty split (its o is not written)
        const float w = exp2f(part - top);
        sum += w;
        const float* o = p.part_o + (i * rows + row) * p.head_dim;
#pragma unroll
        for (int t = 0; t < kMaxDim / 32; ++t)
            if (lane + 32 * t < p.head_dim) acc[t] = fmaf(w, o[lane + 32 * t], acc[t]);
    }
    const float inv = 1.f / sum;
    T* o = static_cast<T*>(p.o) + row * p.head_dim;
#pragma unroll
    for (int t = 0; t < kMaxDim / 32; ++t)
        if (lane + 32 * t < p.head_dim) put(o + lane + 32 * t, acc[t] * inv);
    if (p.lse && lane == 0) p.lse[row] = (top + log2f(sum)) * kRowsLn2;
}

int64_t row_blocks(const GatherProblem& p) {
    const int64_t rows = static_cast<int64_t>(p.total_q) * p.mult * p.heads;
    return (rows + kRowWarps - 1) / kRowWarps;
}

}  // namespace

cudaError_t launch_attn_rows(const GatherProblem& p, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(row_blocks(p)), p.split_keys > 0 ? p.n_splits : 1);
    if (p.kv_lens) attn_rows_kernel<true><<<grid, 32 * kRowWarps, 0, stream>>>(p);
    else attn_rows_kernel<false><<<grid, 32 * kRowWarps, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_attn_join(const GatherProblem& p, int is_bf16, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(row_blocks(p)));
    cfg.blockDim = dim3(32 * kRowWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return is_bf16 ? cudaLaunchKernelEx(&cfg, attn_join_kernel<__nv_bfloat16>, p)
                   : cudaLaunchKernelEx(&cfg, attn_join_kernel<float>, p);
}

}  // namespace pha
