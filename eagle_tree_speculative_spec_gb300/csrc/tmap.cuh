// Host side: TMA tensor maps of row-major matrices.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace e3 {

inline PFN_cuTensorMapEncodeTiled_v12000 tmap_encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *ptr = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return (PFN_cuTensorMapEncodeTiled_v12000)ptr;
        return (PFN_cuTensorMapEncodeTiled_v12000) nullptr;
    }();
    return fn;
}

// `groups` matrices [rows, cols] (2-D without groups), rows ld elements apart and matrices
// group_stride elements apart; boxes of box_rows rows x box_bytes (128 or 64) in the swizzle of that
// width, elements outside a matrix read as zero.  The caller has checked that the base and the pitches are
// multiples of 16 bytes.
inline bool tmap_rows(CUtensorMap *m, CUtensorMapDataType type, int elem_bytes, const void *base, int rows, int cols,
                      int64_t ld, int box_rows, int groups = 0, int64_t group_stride = 0, int box_bytes = 128) {
    const auto fn = tmap_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)(groups > 0 ? groups : 1)};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * elem_bytes, (cuuint64_t)group_stride * elem_bytes};
    const cuuint32_t box[3] = {(cuuint32_t)(box_bytes / elem_bytes), (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, type, groups > 0 ? 3 : 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace e3
