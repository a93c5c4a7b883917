// matvec.cu -- launches of the few-row product with NVFP4 weights (fos_matvec.cuh).
#include "fos_linear_host.cuh"
#include "fos_matvec.cuh"

namespace fos {

namespace {

using namespace matvec;

template <In XT, int kR>
cudaError_t go(MatvecArgs a, const uint8_t* codes, int groups, cudaStream_t s) {
    a.b = codes;
    auto k = k_matvec4<XT, kR>;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem_bytes<kR>());
    if (e != cudaSuccess) return e;
    if (!matrix_map(&a.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, codes, (int64_t)a.G * a.N, a.K / 2, kStepBytes,
                    16 * kR, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.N + 16 * kR - 1) / (16 * kR) * a.splits), (unsigned)groups);
    cfg.blockDim = dim3(32 * kWarpsMv);
    cfg.dynamicSmemBytes = smem_bytes<kR>();
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)a.splits;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k, a);
}

// Row tiles of a CTA and CTAs of a cluster: the pair with the least time, in row
// tiles times steps of a warp, of all CTAs over the device's places (two an SM) and
// half of a last one; what a CTA does once takes as long as eight, its cluster's sums
// as two more.  Measured (us; this pair, the best of the others): 4096 x 14336 1 row
// 12.2 (two tiles, two CTAs), 13.0; 14336 x 4096 8 rows 15.4 (three, one), 17.3;
// eight experts 2048 x 7168 19.9 (four, one), 25.4; six of eight 4096 x 14336 48.6, 57.5 with
// the experts' further rows last (four, one), 49.2 (three, one).
template <In XT>
cudaError_t by_shape(MatvecArgs a, const uint8_t* codes, cudaStream_t s) {
    const int groups = a.ids ? a.M : (a.M + tokens<XT>() - 1) / tokens<XT>();
    const int64_t distinct = a.ids ? (a.M < a.G ? a.M : a.G) : groups;
    const int64_t slots = 2 * (int64_t)sm_count();
    const int nsteps = (a.K + kStepK - 1) / kStepK;
    double least = 1e30;
    int best = 1;
    for (int S = 1; S <= 8; S *= 2) {
        if (S > 1 && nsteps < S * kWarpsMv) break;
        const int steps = ((nsteps + S - 1) / S + kWarpsMv - 1) / kWarpsMv;
        for (int r = 1; r <= 4; ++r) {
            const int64_t ctas = (a.N + 16 * r - 1) / (16 * r) * S * distinct;
            const double one = (r + 0.3) * steps + 8.0 + (S > 1 ? 1.9 : 0.0);
            const double cost = ctas <= slots ? one : one * ((double)ctas / (double)slots + 0.5);
            if (cost < least) {
                least = cost;
                best = r;
                a.splits = S;
            }
        }
    }
    switch (best) {
        case 1: return go<XT, 1>(a, codes, groups, s);
        case 2: return go<XT, 2>(a, codes, groups, s);
        case 3: return go<XT, 3>(a, codes, groups, s);
        default: return go<XT, 4>(a, codes, groups, s);
    }
}

}  // namespace

cudaError_t launch_matvec4(In it, const MatvecArgs& a, const uint8_t* codes, cudaStream_t s) {
    switch (it) {
        case In::BF16: return by_shape<In::BF16>(a, codes, s);
        case In::F16: return by_shape<In::F16>(a, codes, s);
        case In::F32: return by_shape<In::F32>(a, codes, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace fos
