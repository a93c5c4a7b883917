// fos_linear_host.cuh -- launch helpers and TMA descriptors of the product kernels.
#pragma once

#include "fos_linear.cuh"
#include "fos_ops_launch.cuh"
#include "fos_tma_host.cuh"

namespace fos {
namespace lin {

constexpr int kSmemLimit = 232448;  // shared memory of a CTA (227 KiB)

inline bool code_map(CUtensorMap* m, const uint8_t* codes, int64_t rows, int64_t row_bytes, int box_rows) {
    return matrix_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, codes, rows, row_bytes, kRowBytes,
                      box_rows, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// Clusters of `size` CTAs the device holds at once (cached).
template <class Kernel>
int resident_clusters(Kernel k, int threads, int smem, int size) {
    static std::mutex mu;
    static std::unordered_map<LaunchKey, int, LaunchKeyHash> cache;
    const LaunchKey key{reinterpret_cast<const void*>(k), current_device(), threads, (size_t)smem, size};
    std::lock_guard<std::mutex> g(mu);
    auto it = cache.find(key);
    if (it != cache.end()) return it->second;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(size * sm_count()));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)size;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = sm_count() / size;
        if (n < 1) n = 1;
    }
    cache[key] = n;
    return n;
}

template <class Kernel, class Args>
cudaError_t launch_clusters(Kernel k, int clusters, int size, int threads, int smem,
                            const Args& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * size));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)size;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <class F> constexpr int k_tile() { return F::kGlobal ? 64 : 128; }  // K of a scale tile
template <class F> int k_tiles(int64_t K) { return (int)((K + k_tile<F>() - 1) / k_tile<F>()); }
template <class F> int k_stages(int64_t K) { return (k_tiles<F>(K) + F::kSfTiles - 1) / F::kSfTiles; }

// Scale tiles [row tiles, kb, 512 bytes], a box of r x n of them; tiles past
// the ends read as zeros.
inline bool scale_map(CUtensorMap* m, const uint8_t* scales, int64_t rows, int kb, int r, int n) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {kSfTileBytes / 4, (cuuint64_t)kb, (cuuint64_t)((rows + 127) / 128)};
    const cuuint64_t strides[2] = {kSfTileBytes, (cuuint64_t)kb * kSfTileBytes};
    const cuuint32_t box[3] = {kSfTileBytes / 4, (cuuint32_t)n, (cuuint32_t)r};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(scales), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [M, N] of the output's type, box 32 rows x 128 bytes with the 128-byte swizzle.
template <Out OT>
bool chunk_map(CUtensorMap* m, const void* p, int64_t M, int64_t N) {
    constexpr int elt = OT == Out::F32 ? 4 : 2;
    const CUtensorMapDataType dt = OT == Out::F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : OT == Out::F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return matrix_map(m, dt, elt, p, M, N * elt, 128 / elt, 32, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

}  // namespace lin
}  // namespace fos
