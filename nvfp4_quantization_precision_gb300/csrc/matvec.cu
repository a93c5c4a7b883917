// matvec.cu -- launches of the few-row product with NVFP4 weights (fos_matvec.cuh).
#include "fos_matvec.cuh"
#include "fos_ops_launch.cuh"

namespace fos {

namespace {

template <In XT>
cudaError_t go(MatvecArgs a, cudaStream_t s) {
    using namespace matvec;
    const int blocks = (a.N + 127) / 128 * 2;
    const int groups = a.ids ? a.M : (a.M + tokens<XT>() - 1) / tokens<XT>();
    const int distinct = a.ids ? (a.M < a.G ? a.M : a.G) : groups;
    // CTAs of a cluster split K until there are two CTAs an SM; each keeps a step a warp
    const int nsteps = (a.K + kStepK - 1) / kStepK;
    a.splits = 1;
    while (a.splits < 8 && (int64_t)blocks * distinct * a.splits * 2 <= 2 * sm_count() &&
           nsteps >= 2 * a.splits * kWarpsMv)
        a.splits *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * a.splits), (unsigned)groups);
    cfg.blockDim = dim3(32 * kWarpsMv);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)a.splits;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_matvec4<XT>, a);
}

}  // namespace

cudaError_t launch_matvec4(In it, const MatvecArgs& a, cudaStream_t s) {
    switch (it) {
        case In::BF16: return go<In::BF16>(a, s);
        case In::F16: return go<In::F16>(a, s);
        case In::F32: return go<In::F32>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace fos
