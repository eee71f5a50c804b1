// Host-side TMA tensor-map helpers shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fp8fg {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's cuTensorMapEncodeTiled, looked up once through the runtime
// (the library links no driver stub); nullptr when unavailable.
inline EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = []() -> EncodeTiledFn {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// 2-D uint8 tensor [rows][cols] with row pitch `ld` bytes; box
// box_cols x box_rows, 128-byte swizzle. Out-of-range box elements read 0.
inline bool make_map(CUtensorMap *m, const void *base, uint64_t cols, uint64_t rows, uint64_t ld, uint32_t box_cols,
                     uint32_t box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {ld};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Uint8 tensor of rank 3 or 4 over one matrix of row pitch `ld` bytes: `cols`
// contiguous bytes, then dims[i] steps of strides[i] rows each; box box_cols x
// box[0] x ..., 128-byte swizzle, its rows landing one after the other, the
// first of the further dimensions fastest.
inline bool make_map_rows(CUtensorMap *m, const void *base, uint64_t cols, uint64_t ld, int n, const uint64_t *dims,
                          const uint64_t *strides, uint32_t box_cols, const uint32_t *box)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn || n < 1 || n > 3)
        return false;
    cuuint64_t d[4] = {cols, 1, 1, 1}, st[3] = {ld, ld, ld};
    cuuint32_t b[4] = {box_cols, 1, 1, 1}, estr[4] = {1, 1, 1, 1};
    for (int i = 0; i < n; ++i) {
        d[i + 1] = dims[i];
        st[i] = strides[i] * ld;
        b[i + 1] = box[i];
    }
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)(n + 1), const_cast<void *>(base), d, st, b, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D FP32 tensor [rows][cols] with row pitch `ld` elements; box
// box_cols x 1 (one row of scales per copy), no swizzle. Out-of-range box
// elements read 0.
inline bool make_map_f32_row(CUtensorMap *m, const void *base, uint64_t cols, uint64_t rows, uint64_t ld,
                             uint32_t box_cols)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {ld * 4};
    cuuint32_t box[2] = {box_cols, 1};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D bf16 tensor [rows][cols] with row pitch `ld` elements; box
// box_cols x box_rows landing as plain rows (no swizzle). Out-of-range box
// elements read 0.
inline bool make_map_bf16_tile(CUtensorMap *m, const void *base, uint64_t cols, uint64_t rows, uint64_t ld,
                               uint32_t box_cols, uint32_t box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {ld * 2};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace fp8fg
