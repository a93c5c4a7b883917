// fos_ops_launch.cuh -- host-side launch helpers and launcher declarations of
// the feed-forward operators (norm, 8-bit quantization, linear).
#pragma once

#include <cuda_runtime.h>

#include "fos_launch.cuh"

namespace fos {

struct NormArgs;
struct NormBwdArgs;
struct Quant8Args;
struct LinearCall;
enum class Act : int;

// A launch that may be placed while the previous kernel of the stream drains
// (every kernel waits for it before its first global access).
template <class Kernel, class... Args>
inline cudaError_t launch_chained(Kernel kernel, dim3 grid, int threads, size_t smem,
                                  cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Partial rows a column sum may take (rows of its workspace).
constexpr int64_t kMaxParts = 1024;

cudaError_t launch_column_sums(const float* part, int64_t parts, int64_t cols, float* out,
                               cudaStream_t);
cudaError_t launch_rms_norm(In, const NormArgs&, cudaStream_t);
cudaError_t launch_rms_bwd(In, NormBwdArgs, float* dw, float* part, int64_t max_parts,
                           cudaStream_t);
cudaError_t launch_linear(const LinearCall&, cudaStream_t);
cudaError_t launch_quant8(In, Act, const Quant8Args&, cudaStream_t);

}  // namespace fos
