// linear.cu -- launches of the products with an epilogue (fos_linear.cuh).
#include <cstring>

#include "fos_linear.cuh"
#include "fos_linear_pair.cuh"
#include "fos_ops_launch.cuh"
#include "fos_tma_host.cuh"

namespace fos {
namespace lin {

namespace {

constexpr int kSmemLimit = 232448;  // shared memory of a CTA (227 KiB)

bool code_map(CUtensorMap* m, const uint8_t* codes, int64_t rows, int64_t row_bytes, int box_rows) {
    return matrix_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, codes, rows, row_bytes, kRowBytes,
                      box_rows, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// Clusters of `size` CTAs the device holds at once (cached per kernel and size).
template <class Kernel>
int resident_clusters(Kernel k, int threads, int smem, int size) {
    static std::mutex mu;
    static std::unordered_map<uint64_t, int> cache;
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t key = reinterpret_cast<uint64_t>(k) * 64 + (uint64_t)size + ((uint64_t)dev << 56);
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

template <class F, Out OT>
cudaError_t rows_go(const LinearCall& c, cudaStream_t s) {
    RowsArgs a;
    std::memset(&a, 0, sizeof(a));
    const int64_t row_bytes = F::kGlobal ? c.K / 2 : c.K;
    a.nt = c.M >= 256 ? 256 : (int)((c.M + 15) / 16 * 16);
    if (!code_map(&a.tp, c.b, c.N, row_bytes, 128) || !code_map(&a.tq, c.a, c.M, row_bytes, a.nt))
        return cudaErrorInvalidValue;
    a.sfp = c.bs;
    a.sfq = c.as;
    a.ep = c.ep;
    a.M = c.M;
    a.N = c.N;
    const int blk4 = F::kGlobal ? 64 : 128;
    a.kb = (int)((c.K + blk4 - 1) / blk4);
    a.nkb = (a.kb + F::kSfTiles - 1) / F::kSfTiles;
    a.tiles_p = (int)((c.N + 127) / 128);
    a.tiles = a.tiles_p * (int)((c.M + a.nt - 1) / a.nt);
    const int stage = rows_stage_bytes<F>(a.nt);
    a.stages = (kSmemLimit - 3072) / stage;
    if (a.stages > kMaxStages) a.stages = kMaxStages;
    const int smem = a.stages * stage + 1024;
    auto k = k_linear_rows<F, OT>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), (size_t)kSmemLimit - 2048);
    if (e != cudaSuccess) return e;
    // the split of K that needs the fewest rounds of the device, counted in
    // whole-K tiles; every CTA keeps at least two stages
    int best = 1, clusters = sm_count();
    double cost = 1e30;
    for (int S = 1; S <= 8; S *= 2) {
        if (S > 1 && a.nkb / S < 2) break;
        const int fit = S == 1 ? sm_count() : resident_clusters(k, kRowsThreads, smem, S);
        const double t = (double)((a.tiles + fit - 1) / fit) / S;
        if (t < 0.95 * cost) {
            cost = t;
            best = S;
            clusters = fit;
        }
    }
    a.splits = best;
    if (clusters > a.tiles) clusters = a.tiles;
    return launch_clusters(k, clusters, best, kRowsThreads, smem, a, s);
}

// Scale tiles [row tiles, kb, 512 bytes], a box of r x n of them; tiles past
// the ends read as zeros.
bool scale_map(CUtensorMap* m, const uint8_t* scales, int64_t rows, int kb, int r, int n) {
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

template <class F, Out OT>
cudaError_t pair_go(const LinearCall& c, cudaStream_t s) {
    PairArgs a;
    std::memset(&a, 0, sizeof(a));
    const int64_t row_bytes = F::kGlobal ? c.K / 2 : c.K;
    const int blk4 = F::kGlobal ? 64 : 128;
    a.kb = (int)((c.K + blk4 - 1) / blk4);
    a.nkb = (a.kb + F::kSfTiles - 1) / F::kSfTiles;
    if (!code_map(&a.ta, c.a, c.M, row_bytes, 128) || !code_map(&a.tb, c.b, c.N, row_bytes, 96) ||
        !scale_map(&a.tsa, c.as, c.M, a.kb, 1, kSfChunkTiles) ||
        !scale_map(&a.tsb, c.bs, c.N, a.kb, 2, kSfChunkTiles) ||
        !chunk_map<OT>(&a.tout, c.ep.out, c.M, c.N) ||
        (c.ep.residual && !chunk_map<OT>(&a.tres, c.ep.residual, c.M, c.N)) ||
        (c.ep.pre && !chunk_map<OT>(&a.tpre, c.ep.pre, c.M, c.N)))
        return cudaErrorInvalidValue;
    a.ep = c.ep;
    a.M = c.M;
    a.N = c.N;
    a.tiles_m = (int)((c.M + kPairM - 1) / kPairM);
    a.tiles_n = (int)((c.N + kPairN - 1) / kPairN);
    a.bufs = c.ep.pre ? 4 : 2;
    const int other = 4 * a.bufs * kChunkBytes + kSfSlots * kSfChunkBytes + 4 * kPairN * 4;
    a.stages = (kSmemLimit - 2048 - other) / kPairStageBytes;
    const int smem = a.stages * kPairStageBytes + other + 1024;
    auto k = k_linear_pair<F, OT>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), (size_t)kSmemLimit - 1024);
    if (e != cudaSuccess) return e;
    const int tiles = a.tiles_m * a.tiles_n;
    int clusters = resident_clusters(k, kPairThreads, smem, 2);
    if (clusters > tiles) clusters = tiles;
    return launch_clusters(k, clusters, 2, kPairThreads, smem, a, s);
}

template <class F, Out OT>
cudaError_t go(const LinearCall& c, cudaStream_t s) {
    return c.M > 256 ? pair_go<F, OT>(c, s) : rows_go<F, OT>(c, s);
}

template <class F>
cudaError_t by_out(const LinearCall& c, cudaStream_t s) {
    switch (c.out) {
        case In::BF16: return go<F, Out::BF16>(c, s);
        case In::F16: return go<F, Out::F16>(c, s);
        case In::F32: return go<F, Out::F32>(c, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace lin

cudaError_t launch_linear(const LinearCall& c, cudaStream_t s) {
    return c.fmt4 ? lin::by_out<lin::F4>(c, s) : lin::by_out<lin::F8>(c, s);
}

}  // namespace fos
