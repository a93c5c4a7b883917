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

// Shape of a rows launch and what it should take.
struct RowsPlan {
    int nt, stages, smem, splits, clusters;
    double us;
};

// Both kernels' times by sizes, from measurements over 1 .. 1024 tokens, 1024 ..
// 14336 weight rows and K of 4096 and 14336 (us; 8 bit, NVFP4):
//   rows  (4.2, 4.5) + rounds (stages / S (0.32, 0.37 + 0.00043 nt) + 0.022 nt,
//         0.034 without a split)
//   pair  6.1 + the larger of rounds * stages (0.225, 0.29) and the weights at
//         (5.6, 4.7) TB/s
// E.g. 8 bit, 4096 x 14336: 64 tokens 15.7 rows, 31.0 pair; 256 tokens 22.6 and
// 31.5.  14336 x 4096: 32 tokens 15.1 and 16.3; 256 tokens 26.5 and 17.5 (NVFP4
// 10.6 and 13.5, 19.0 and 13.7).  Checked over 216 sizes with K of 512 .. 16384: the
// kernel taken is within 10 % of the faster one in 205, at worst 39 % (64 tokens, K =
// 512: 6.2 and 4.5 us, the rows kernel's fixed part being less there).
template <class F, Out OT>
RowsPlan rows_plan(const LinearCall& c) {
    // The wait for the stage that used a scale buffer last may look back one turn
    // of the ring at most (a full tile of tokens has the fewest stages).
    static_assert((kSmemLimit - 3 * 1024) / rows_stage_bytes<F>(256) >= kSfRing && kMaxStages >= kSfRing,
                  "stages");
    RowsPlan p;
    p.nt = c.M >= 256 ? 256 : (int)((c.M + 15) / 16 * 16);
    const int stage = rows_stage_bytes<F>(p.nt);
    p.stages = (kSmemLimit - 3 * 1024) / stage;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    p.smem = p.stages * stage + 1024;
    const int nkb = k_stages<F>(c.K);
    const int64_t tiles = (c.N + 127) / 128 * ((c.M + p.nt - 1) / p.nt);
    // the split of K with the shortest time; every CTA keeps at least two stages
    p.us = 1e30;
    for (int S = 1; S <= 8 && (S == 1 || nkb / S >= 2); S *= 2) {
        const int fit = S == 1 ? sm_count()
                               : resident_clusters(k_linear_rows<F, OT>, kRowsThreads, p.smem, S);
        const double stage_us = (F::kGlobal ? 0.37 : 0.32) + 0.00043 * p.nt;
        const double us = (F::kGlobal ? 4.5 : 4.2) + (double)((tiles + fit - 1) / fit) *
                              ((nkb + S - 1) / S * stage_us + (S > 1 ? 0.022 : 0.034) * p.nt);
        if (us < p.us) {
            p.us = us;
            p.splits = S;
            p.clusters = fit < tiles ? fit : (int)tiles;
        }
    }
    return p;
}

template <class F>
double pair_us(const LinearCall& c) {
    const int64_t tiles = (c.M + kPairM - 1) / kPairM * ((c.N + kPairN - 1) / kPairN);
    const int64_t pairs = sm_count() / 2;
    const double work = (double)((tiles + pairs - 1) / pairs) * k_stages<F>(c.K) *
                        (F::kGlobal ? 0.29 : 0.225);
    const double weights = (double)c.N * c.K * (F::kGlobal ? 0.5625 / 4.7e6 : 1.03125 / 5.6e6);
    return 6.1 + (work > weights ? work : weights);
}

template <class F, Out OT>
cudaError_t rows_go(const LinearCall& c, const RowsPlan& p, cudaStream_t s) {
    RowsArgs a;
    std::memset(&a, 0, sizeof(a));
    const int64_t row_bytes = F::kGlobal ? c.K / 2 : c.K;
    a.nt = p.nt;
    if (!code_map(&a.tp, c.b, c.N, row_bytes, 128) || !code_map(&a.tq, c.a, c.M, row_bytes, a.nt))
        return cudaErrorInvalidValue;
    a.sfp = c.bs;
    a.sfq = c.as;
    a.ep = c.ep;
    a.M = c.M;
    a.N = c.N;
    a.kb = k_tiles<F>(c.K);
    a.nkb = k_stages<F>(c.K);
    a.tiles_p = (int)((c.N + 127) / 128);
    a.tiles = a.tiles_p * (int)((c.M + a.nt - 1) / a.nt);
    a.stages = p.stages;
    a.splits = p.splits;
    return launch_clusters(k_linear_rows<F, OT>, p.clusters, p.splits, kRowsThreads, p.smem, a, s);
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
    a.kb = k_tiles<F>(c.K);
    a.nkb = k_stages<F>(c.K);
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
    // Bands of equal height whose rows of a take at most 30 MB, a quarter of L2: they
    // stay there while b streams past once a band.  Under load, against bands of 8
    // always: 8 bit 8192 x 14336 x 4096 (16 rows) 355 and 364 us, NVFP4 the same (32)
    // 180 and 184; 8 bit 8192 x 4096 x 14336 (8) 327, with 16 331 and with 32 356.
    const int fit = (int)(30000000 / (kPairM * row_bytes));
    const int bands = (a.tiles_m + (fit > 1 ? fit : 1) - 1) / (fit > 1 ? fit : 1);
    a.band = (a.tiles_m + bands - 1) / bands;
    a.bufs = c.ep.pre ? 4 : 2;
    const int other = 4 * a.bufs * kChunkBytes + sf_slots<F>() * kSfChunkBytes + 4 * kPairN * 4;
    static_assert((kSmemLimit - 2048 - 16 * kChunkBytes - kSfMaxSlots * kSfChunkBytes - 16 * kPairN) /
                          kPairStageBytes >= kSfBufs, "stages");
    a.stages = (kSmemLimit - 2048 - other) / kPairStageBytes;
    const int smem = a.stages * kPairStageBytes + other + 1024;
    auto k = k_linear_pair<F, OT>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), (size_t)kSmemLimit - 1024);
    if (e != cudaSuccess) return e;
    const int tiles = a.tiles_m * a.tiles_n;
    int clusters = resident_clusters(k, pair_threads<F>(), smem, 2);
    if (clusters > tiles) clusters = tiles;
    return launch_clusters(k, clusters, 2, pair_threads<F>(), smem, a, s);
}

template <class F, Out OT>
cudaError_t go(const LinearCall& c, cudaStream_t s) {
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k_linear_rows<F, OT>),
                                     (size_t)kSmemLimit - 2048);
    if (e != cudaSuccess) return e;
    const RowsPlan p = rows_plan<F, OT>(c);
    return p.us <= pair_us<F>(c) ? rows_go<F, OT>(c, p, s) : pair_go<F, OT>(c, s);
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
