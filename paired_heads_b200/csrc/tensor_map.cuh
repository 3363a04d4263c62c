// tensor_map.cuh -- TMA tensor maps over the slot view of a caller's buffer.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

namespace pha {

inline PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
    // Resolved through the runtime so that the library does not link libcuda directly.
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
}

// 2-D bf16 map over [rows][width] elements, box 64 x box_rows, 128-byte swizzle, zero fill
// outside.
inline bool encode_slot_map(CUtensorMap* map, const void* base, uint64_t width, uint64_t rows,
                     uint32_t box_rows = 128) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = get_encode();
    if (!encode) return false;
    cuuint64_t dims[2] = {width, rows};
    cuuint64_t strides[1] = {width * 2};
    cuuint32_t box[2] = {64, box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// 2-D uint8 map over [rows][width] bytes for e4m3 tiles: box box_inner x 128, swizzled to match
// the box width (128-byte rows: 128-byte swizzle; 64-byte rows: 64-byte swizzle) or unswizzled.
inline bool encode_u8_map(CUtensorMap* map, const void* base, uint64_t width, uint64_t rows,
                   uint32_t box_inner, bool swizzle) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = get_encode();
    if (!encode) return false;
    cuuint64_t dims[2] = {width, rows};
    cuuint64_t strides[1] = {width};
    cuuint32_t box[2] = {box_inner, 128};
    cuuint32_t estr[2] = {1, 1};
    const CUtensorMapSwizzle sw = !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE
                                  : box_inner == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                                     : CU_TENSOR_MAP_SWIZZLE_64B;
    CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// 3-D bf16 map over q [rows][heads][hd] whose box is 64 columns of `pack` heads of 128 / pack rows (pack
// divides 128): a query tile with its rows in (row, head) order. 128-byte swizzle, zero fill outside.
inline bool encode_pack_map(CUtensorMap* map, const void* base, uint64_t hd, uint64_t heads, uint64_t rows,
                            uint32_t pack) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = get_encode();
    if (!encode) return false;
    cuuint64_t dims[3] = {hd, heads, rows};
    cuuint64_t strides[2] = {hd * 2, heads * hd * 2};
    cuuint32_t box[3] = {64, pack, 128 / pack};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

}  // namespace pha
