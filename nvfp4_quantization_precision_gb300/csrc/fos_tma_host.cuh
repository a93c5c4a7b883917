// fos_tma_host.cuh -- TMA descriptors on the host.
#pragma once

#include <cudaTypedefs.h>

#include <mutex>

#include <cuda_runtime.h>

namespace fos {

// cuTensorMapEncodeTiled is a driver function; its address comes from the
// runtime once (no link against the driver library).
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        else
            cudaGetLastError();
    });
    return fn;
}

// A row-major [rows, row_bytes] matrix of `dt` elements of `elt` bytes as a 2D
// tensor with boxes of box_x elements x box_rows rows; what a box reads past
// the ends is zero.  row_bytes is a multiple of 16.
inline bool matrix_map(CUtensorMap* map, CUtensorMapDataType dt, int elt, const void* p,
                       int64_t rows, int64_t row_bytes, int box_x, int box_rows,
                       CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promotion) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)(row_bytes / elt), (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
    const cuuint32_t box[2] = {(cuuint32_t)box_x, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, dt, 2, const_cast<void*>(p), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promotion,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace fos
