// attn_decode.cu -- bf16 attention of few new tokens per sequence over a paged cache (decoding): up to
// 16 query rows (tokens times the heads of a kv head's group) against a long run of keys.
//
// What it has to do is read every visible key row once, K and V; the products are 2 x 16 x hd
// multiply-adds a key, far below what that takes. So the kernel is built around copies in flight: a
// block per (key range, kv head, sequence), each of its 4 warps streaming its own 16-key steps through
// a private ring of shared-memory stages (16-byte cp.async straight from the page rows; no barrier
// between warps in the loop), 2 blocks of 96 KB per SM at hd 128 (128 KB in flight). Tensor memory and
// the M = 128 products of attn_gather.cu would need the set-up of a large tile for 16 rows: 242 us
// against 176 us here, 6.2 TB/s (64 single tokens over ragged histories of up to 8192, 32 / 8 heads of 128).
//
// Per step: S = Q K^T by m16n8k16 (Q in registers for the whole range), the running maximum and sum per
// row (four lanes share a row), P rounded to bf16 as the A operand of O += P V; O in registers. At the
// end the four warps' parts are joined through shared memory; a sequence longer than one range leaves
// partial rows for attn_join_kernel.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gather.cuh"

namespace pha {

namespace {

constexpr int kWarps = 4;
constexpr int kStepKeys = 16;
constexpr int kStages = 3;
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2F = 0.6931471805599453f;

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// D += A B, m16n8k16, bf16 inputs, float32 accumulation.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int HD>
constexpr int stage_bytes() { return 2 * kStepKeys * HD * 2; }
template <int HD>
constexpr int smem_bytes() { return kWarps * kStages * stage_bytes<HD>(); }

template <int HD>
__global__ void __launch_bounds__(32 * kWarps) attn_decode_kernel(const GatherProblem p) {
    constexpr int kUnits = HD / 8, kRpi = 32 / kUnits;  // 16-byte units of a row, rows per copy instruction
    constexpr int kRowBytes = HD * 2;
    static_assert(kStages * stage_bytes<HD>() >= 16 * HD * 4, "a warp's partial O fits its stages");
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float part_m[kWarps][16], part_l[kWarps][16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.z, g = blockIdx.y, split = blockIdx.x;
    const GatherSeq s = gather_seq(p, b);
    if (!s.ok) {
        if (p.status && threadIdx.x == 0) atomicMax(p.status, DEV_BAD_SEQLENS);
        return;
    }
    if (s.n_q == 0) return;
    const int pos0 = s.kv - s.n_q;
    const GatherCols cols = gather_cols(p, pos0, s.n_q);
    const int c0 = split * p.split_keys;
    if (c0 >= cols.total) return;
    const int c1 = c0 + p.split_keys < cols.total ? c0 + p.split_keys : cols.total;
    const int G = p.heads / p.kv_heads;
    const int n_rows = s.n_q * G;
    const int steps = (c1 - c0 + kStepKeys - 1) / kStepKeys;

    const uint32_t ring = smem_u32(smem) + warp * kStages * stage_bytes<HD>();
    const int unit = lane % kUnits;
    const __nv_bfloat16* k_all = static_cast<const __nv_bfloat16*>(p.k) + static_cast<int64_t>(g) * HD + unit * 8;
    const __nv_bfloat16* v_all = static_cast<const __nv_bfloat16*>(p.v) + static_cast<int64_t>(g) * HD + unit * 8;
    const int64_t stride = static_cast<int64_t>(p.kv_heads) * HD;
    // The table entry of this lane's key of a step, read one step ahead of the copies that need it.
    auto entry_of = [&](int step) -> int {
        const int col = c0 + step * kStepKeys + (lane & 15);
        if (col >= c1) return -1;
        return __ldg(p.table + static_cast<int64_t>(b) * p.max_pages + (col_pos(cols, col) >> p.page_shift));
    };
    int entry = entry_of(warp);
    // copies of step `step` (the next one that `entry` is for) into stage `st`: one group, empty past the
    // last step
    auto fetch = [&](int step, int st) {
        if (step < steps) {
            const int col = c0 + step * kStepKeys + (lane & 15);
            const int page = entry;
            entry = entry_of(step + kWarps);
            const bool is_page = page >= 0 && page < p.n_pages;
            if (col < c1 && !is_page && p.status) atomicMax(p.status, DEV_BAD_PAGE);
            const int in = col_pos(cols, col) & ((1 << p.page_shift) - 1);
            const int mine = col < c1 && is_page ? (page << p.page_shift) + in : -1;
            const uint32_t k_st = ring + st * stage_bytes<HD>(), v_st = k_st + kStepKeys * kRowBytes;
#pragma unroll
            for (int i = 0; i < kStepKeys / kRpi; ++i) {
                const int r = i * kRpi + lane / kUnits;
                const int x = __shfl_sync(0xffffffffu, mine, r);
                const int64_t at = (x < 0 ? 0 : x) * stride;
                const uint32_t to = r * kRowBytes + ((unit ^ (r & 7)) << 4);
                cp_async_16_zfill(k_st + to, k_all + at, x < 0 ? 0u : 16u);
                cp_async_16_zfill(v_st + to, v_all + at, x < 0 ? 0u : 16u);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(warp + i * kWarps, i);

    // Q fragments: rows lane / 4 and lane / 4 + 8 of the 16 (row = token * G + head), zeros past n_rows
    uint32_t qa[HD / 16][4];
    const int row_a = lane >> 2, row_b = row_a + 8;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + static_cast<int64_t>(g) * G * HD + 2 * (lane & 3);
    auto q_row = [&](int row) {
        return q + ((s.q0 + row / G) * p.heads + row % G) * HD;
    };
    const __nv_bfloat16 *qa_row = q_row(row_a < n_rows ? row_a : 0), *qb_row = q_row(row_b < n_rows ? row_b : 0);
#pragma unroll
    for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t a = __ldg(reinterpret_cast<const uint32_t*>(qa_row + 16 * ks + 8 * h));
            const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(qb_row + 16 * ks + 8 * h));
            qa[ks][2 * h] = row_a < n_rows ? a : 0u;
            qa[ks][2 * h + 1] = row_b < n_rows ? c : 0u;
        }
    const int pos_a = pos0 + row_a / G, pos_b = pos0 + row_b / G;
    const float scale2 = p.scale * kLog2E;
    float o[HD / 8][4];
#pragma unroll
    for (int n = 0; n < HD / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // of rows a, b; l of this lane's columns

    // Columns that some row does not see: below n_q - 1 (the window's start moves with the row) and the last
    // n_q - 1 of the window part. Only steps with one of them, or with the range's end, take the mask
    // (every step of two new slots: 53 us instead of 35, 32 paired sequences of 4,106 visible keys).
    const int all_from = p.window > 0 ? s.n_q - 1 : 0, all_to = cols.n_w - (s.n_q - 1);
    int st = 0;
    for (int step = warp; step < steps; step += kWarps) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        const uint32_t k_st = ring + st * stage_bytes<HD>(), v_st = k_st + kStepKeys * kRowBytes;
        float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        {
            const int key = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
            const uint32_t row_at = k_st + key * kRowBytes;
#pragma unroll
            for (int ks = 0; ks < HD / 16; ++ks) {
                uint32_t kb[4];
                ldsm4(row_at + (((2 * ks + half) ^ (key & 7)) << 4), kb);
                mma_bf16(sc[0], qa[ks], kb[0], kb[1]);
                mma_bf16(sc[1], qa[ks], kb[2], kb[3]);
            }
        }
        // scaled scores, -inf where hidden; then the rows' maxima over their four lanes
        const int col = c0 + step * kStepKeys + 2 * (lane & 3);
        float mx[2] = {-INFINITY, -INFINITY};
        const int first = c0 + step * kStepKeys, past = first + kStepKeys;
        const bool edge = past > c1 || first < all_from || (past > all_to && first < cols.n_w);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = sc[n][e] * scale2;
                if (edge) {
                    const int c = col + 8 * n + (e & 1);
                    if (c >= c1 || !col_visible(p, cols, c, e < 2 ? pos_a : pos_b)) x = -INFINITY;
                }
                sc[n][e] = x;
                mx[e >> 1] = fmaxf(mx[e >> 1], x);
            }
        bool grown = false;
        float alpha[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
            // the reference stays until the maximum has grown by more than 2^8 (any reference is exact)
            const bool up = mx[h] > m[h] + 8.f;
            alpha[h] = up ? ex2(m[h] - mx[h]) : 1.f;
            m[h] = up ? mx[h] : m[h];
            grown |= up;
        }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int n = 0; n < HD / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][e] *= alpha[e >> 1];
        }
        const float neg_a = m[0] == -INFINITY ? 0.f : -m[0], neg_b = m[1] == -INFINITY ? 0.f : -m[1];
        float w[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) w[n][e] = ex2(sc[n][e] + (e < 2 ? neg_a : neg_b));
        l[0] = l[0] * alpha[0] + ((w[0][0] + w[0][1]) + (w[1][0] + w[1][1]));
        l[1] = l[1] * alpha[1] + ((w[0][2] + w[0][3]) + (w[1][2] + w[1][3]));
        // the weights are rounded to bf16 for the tensor cores; their sum keeps float32
        const uint32_t pa[4] = {pack_bf16x2(w[0][0], w[0][1]), pack_bf16x2(w[0][2], w[0][3]),
                                pack_bf16x2(w[1][0], w[1][1]), pack_bf16x2(w[1][2], w[1][3])};
        {
            const int key = (lane & 7) + (((lane >> 3) & 1) << 3), half = lane >> 4;
            const uint32_t row_at = v_st + key * kRowBytes;
#pragma unroll
            for (int n = 0; n < HD / 8; n += 2) {
                uint32_t vb[4];
                ldsm4_trans(row_at + (((n + half) ^ (key & 7)) << 4), vb);
                mma_bf16(o[n], pa, vb[0], vb[1]);
                mma_bf16(o[n + 1], pa, vb[2], vb[3]);
            }
        }
        __syncwarp();  // every lane is done with the stage that is filled next
        fetch(step + (kStages - 1) * kWarps, st == 0 ? kStages - 1 : st - 1);
        st = st + 1 == kStages ? 0 : st + 1;
    }
    cp_async_wait<0>();
    __syncwarp();
    // this warp's part into its stages
    float* po = reinterpret_cast<float*>(smem + warp * kStages * stage_bytes<HD>());
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        const int row = h ? row_b : row_a;
        if ((lane & 3) == 0) {
            part_m[warp][row] = m[h];
            part_l[warp][row] = l[h];
        }
        if (row < n_rows)
#pragma unroll
            for (int n = 0; n < HD / 8; ++n)
                *reinterpret_cast<float2*>(po + row * HD + 8 * n + 2 * (lane & 3)) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
    }
    __syncthreads();
    const bool alone = cols.total <= p.split_keys;
    const int64_t all_rows = static_cast<int64_t>(p.total_q) * p.mult * p.heads;
    for (int row = warp; row < n_rows; row += kWarps) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) top = fmaxf(top, part_m[i][row]);
        float sum = 0.f, acc[HD / 32];
#pragma unroll
        for (int e = 0; e < HD / 32; ++e) acc[e] = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (part_l[i][row] == 0.f) continue;  // nothing visible in this warp's steps
            const float w = ex2(part_m[i][row] - top);
            sum = fmaf(w, part_l[i][row], sum);
            const float* from = reinterpret_cast<const float*>(smem + i * kStages * stage_bytes<HD>()) + row * HD;
#pragma unroll
            for (int e = 0; e < HD / 32; ++e) acc[e] = fmaf(w, from[32 * e + lane], acc[e]);
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const int64_t out = (s.q0 + row / G) * p.heads + g * G + row % G;
        if (alone) {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + out * HD;
#pragma unroll
            for (int e = 0; e < HD / 32; ++e) dst[32 * e + lane] = __float2bfloat16_rn(acc[e] * inv);
            if (p.lse && lane == 0) p.lse[out] = (top + log2f(sum)) * kLn2F;
        } else {
            float* dst = p.part_o + (split * all_rows + out) * HD;
#pragma unroll
            for (int e = 0; e < HD / 32; ++e) dst[32 * e + lane] = acc[e] * inv;
            if (lane == 0) p.part_lse[split * all_rows + out] = sum != 0.f ? top + log2f(sum) : -INFINITY;  // (NaN stays)
        }
    }
}

template <int HD>
cudaError_t launch_decode_hd(const GatherProblem& p, cudaStream_t stream) {
    const cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               smem_bytes<HD>());
    if (e != cudaSuccess) return e;
    attn_decode_kernel<HD><<<dim3(p.n_splits, p.kv_heads, p.batch), 32 * kWarps, smem_bytes<HD>(), stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_decode(const GatherProblem& p, cudaStream_t stream) {
    if (p.head_dim == 128) return launch_decode_hd<128>(p, stream);
    if (p.head_dim == 64) return launch_decode_hd<64>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pha
