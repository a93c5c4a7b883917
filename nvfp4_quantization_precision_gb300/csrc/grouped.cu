// grouped.cu -- launches of the products grouped by expert (fos_grouped.cuh).
#include <cstring>

#include "fos_grouped.cuh"
#include "fos_grouped_rows.cuh"
#include "fos_linear_host.cuh"

namespace fos {
namespace lin {

namespace {

// `own`: bytes left for the kernel's static shared memory.
template <class Kernel, class Args>
cudaError_t launch_pairs(Kernel k, int own, int threads, int64_t tiles, int smem, const Args& a, cudaStream_t s) {
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), (size_t)(kSmemLimit - own));
    if (e != cudaSuccess) return e;
    int64_t clusters = resident_clusters(k, threads, smem, 2);
    if (clusters > tiles) clusters = tiles;
    return launch_clusters(k, (int)clusters, 2, threads, smem, a, s);
}

// Which of the two products, by models of their times (us) for the routing that the
// host can know: as many experts with rows as there can be, `mean` rows each.
//   k_grouped_rows  5.0 + rounds (stages / S (0.32, NVFP4 0.37, + 0.00043 nt) + 0.022 mean,
//                   0.034 without a split) + 4.0 (1.2 without a split) a further round,
//                   whose first stages come after the last round's sums
//   k_grouped       6.0 + turns x stages (0.21 + 0.00025 mean, NVFP4 0.36; 0.0036 mean more
//                   where the tokens' scales come by cp.async)
// The former is taken where it should need at most 0.85 of the other's time. Measured
// (rows, k_grouped; * taken): 8 bit, 2 rows of 2 of 17 experts x 320 x 8192 7.4*, 18.3; 855 rows
// of 2 x 368 x 15360 26.0*, 36.4; 300 of 8 x 1024 x 4096 16.7, 13.8*; 8 of 6 of 8 x
// 14336 x 4096 68.1, 59.9*; NVFP4, 256 of 4 x 1024 x 8192 12.1*, 15.5; 16 of 8 of 16 x 2048 x 7168
// 15.7, 16.4*; 128 of 54 of 64 x 2048 x 7168 79.9, 71.5*.  Of 32 sizes the one taken was
// slower than the other in seven, by 1 us at most.
struct GroupedRowsPlan {
    int nt, stages, smem, splits, clusters;
    double us;
};

double mean_rows(const GroupedCall& c, int most) {
    const double mean = (double)c.rows / (double)(c.rows < c.G ? c.rows : c.G);
    return mean < most ? mean : most;
}
template <class F>
double grouped_us(const GroupedCall& c) {
    const int64_t tiles = (c.N + kPairM - 1) / kPairM * group_tiles_max(c.rows, c.G, kTokTile);
    const int64_t pairs = sm_count() / 2;
    const double mean = mean_rows(c, kTokTile);
    const bool wide = (c.K / (F::kGlobal ? 16 : 32)) % 16 == 0;
    const double stage = (F::kGlobal ? 0.36 : 0.21 + 0.00025 * mean) + (wide ? 0.0 : 0.0036 * mean);
    return 6.0 + (double)((tiles + pairs - 1) / pairs) * k_stages<F>(c.K) * stage;
}

constexpr int kRowsOwn = 2048;
template <class F, Out OT>
GroupedRowsPlan grouped_rows_plan(const GroupedCall& c) {
    GroupedRowsPlan p;
    p.nt = c.rows >= kGrpRowsTok ? kGrpRowsTok : (int)((c.rows + 15) / 16 * 16);
    const int stage = rows_stage_bytes<F>(p.nt), table = (int)group_table_bytes(c.G);
    static_assert((kSmemLimit - kRowsOwn - 1024 - (int)group_table_bytes(kMaxGroups)) / rows_stage_bytes<F>(kGrpRowsTok) >=
                      kSfRing, "stages");
    p.stages = (kSmemLimit - kRowsOwn - 1024 - table) / stage;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    p.smem = p.stages * stage + table + 1024;
    const int nkb = k_stages<F>(c.K);
    // most experts that can have rows, each with a chunk begun
    const int64_t tiles = (c.N + 127) / 128 * group_tiles_max(c.rows, c.G, kGrpRowsTok);
    const double mean = mean_rows(c, kGrpRowsTok);
    p.us = 1e30;
    for (int S = 1; S <= 8 && (S == 1 || nkb / S >= 2); S *= 2) {
        const int fit = S == 1 ? sm_count() : resident_clusters(k_grouped_rows<F, OT>, kRowsThreads, p.smem, S);
        const double stage_us = (F::kGlobal ? 0.37 : 0.32) + 0.00043 * p.nt;
        const double rounds = (double)((tiles + fit - 1) / fit);
        const double us = 5.0 + rounds * ((nkb + S - 1) / S * stage_us + (S > 1 ? 0.022 : 0.034) * mean) +
                          (rounds - 1.0) * (S > 1 ? 4.0 : 1.2);
        if (us < p.us) {
            p.us = us;
            p.splits = S;
            p.clusters = fit < tiles ? fit : (int)tiles;
        }
    }
    return p;
}

template <class F, Out OT>
cudaError_t rows_go(const GroupedCall& c, const GroupedRowsPlan& p, cudaStream_t s) {
    GroupedRowsArgs a;
    std::memset(&a, 0, sizeof(a));
    const int64_t row_bytes = F::kGlobal ? c.K / 2 : c.K;
    a.nt = p.nt;
    if (!code_map(&a.tp, c.b, c.G * c.N, row_bytes, 128) || !code_map(&a.tq, c.a, c.rows, row_bytes, a.nt))
        return cudaErrorInvalidValue;
    a.sfp = c.bs;
    a.sfq = c.as;
    a.sfq_pitch = F::kGlobal ? c.K / 16 : c.K / 32;
    a.ep = c.ep;
    a.offs = c.offs;
    a.G = c.G;
    a.rows = (int)c.rows;
    a.N = (int)c.N;
    a.tiles_p = (int)((c.N + 127) / 128);
    a.kb = k_tiles<F>(c.K);
    a.nkb = k_stages<F>(c.K);
    a.stages = p.stages;
    a.splits = p.splits;
    return launch_clusters(k_grouped_rows<F, OT>, p.clusters, p.splits, kRowsThreads, p.smem, a, s);
}

template <class F, Out OT>
cudaError_t go(const GroupedCall& c, cudaStream_t s) {
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k_grouped_rows<F, OT>), (size_t)(kSmemLimit - kRowsOwn));
    if (e != cudaSuccess) return e;
    const GroupedRowsPlan plan = grouped_rows_plan<F, OT>(c);
    if (plan.us < 0.85 * grouped_us<F>(c)) return rows_go<F, OT>(c, plan, s);
    GroupedArgs a;
    std::memset(&a, 0, sizeof(a));
    const int64_t row_bytes = F::kGlobal ? c.K / 2 : c.K;
    a.kb = k_tiles<F>(c.K);
    a.nkb = k_stages<F>(c.K);
    a.row_tiles = (int)((c.N + 127) / 128);
    if (!code_map(&a.tw, c.b, c.G * c.N, row_bytes, 128) || !code_map(&a.tt, c.a, c.rows, row_bytes, kTokTile / 2) ||
        !code_map(&a.tt16, c.a, c.rows, row_bytes, kTokBox) ||
        !scale_map(&a.tsw, c.bs, (int64_t)c.G * a.row_tiles * 128, a.kb, 1, kSfChunkTiles))
        return cudaErrorInvalidValue;
    a.ep = c.ep;
    a.ts = c.as;
    a.ts_pitch = F::kGlobal ? c.K / 16 : c.K / 32;
    a.ts_wide = a.ts_pitch % 16 == 0;
    if (a.ts_wide && (!matrix_map(&a.tst, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, c.as, c.rows, a.ts_pitch, 16, kTokTile,
                                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_64B) ||
                      !matrix_map(&a.tst32, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, c.as, c.rows, a.ts_pitch, 16, 32,
                                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_64B)))
        return cudaErrorInvalidValue;
    a.offs = c.offs;
    a.G = c.G;
    a.rows = (int)c.rows;
    a.N = (int)c.N;
    a.tiles_n = (int)((c.N + kPairM - 1) / kPairM);
    a.band = token_band(c.rows, row_bytes);
    constexpr int kOwn = 8192;
    constexpr int kFixed = kOwn + 1024 + grp_slots<F>() * kGrpSfBytes;
    constexpr int kRes = 8 * grp_res_slots<OT>() * grp_res_bytes<OT>();
    static_assert((kSmemLimit - kFixed - kRes - (int)group_table_bytes(kMaxGroups)) / kPairStageBytes >= kSfBufs, "stages");
    if (c.ep.residual) {
        constexpr int kElt = OT == Out::F32 ? 4 : 2;
        constexpr CUtensorMapDataType kType = OT == Out::F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                              : OT == Out::F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                               : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        if (!matrix_map(&a.tres, kType, kElt, c.ep.residual, c.rows, c.N * kElt, 32, kEpiTok, CU_TENSOR_MAP_SWIZZLE_NONE,
                        CU_TENSOR_MAP_L2_PROMOTION_NONE))
            return cudaErrorInvalidValue;
    }
    a.res_area = c.ep.residual ? kRes : 0;
    const int other = grp_slots<F>() * kGrpSfBytes + a.res_area + (int)group_table_bytes(c.G);
    a.stages = (kSmemLimit - kOwn - 1024 - other) / kPairStageBytes;
    if (a.stages > kPairMaxStages) a.stages = kPairMaxStages;
    const int smem = a.stages * kPairStageBytes + other + 1024;
    return launch_pairs(k_grouped<F, OT>, kOwn, grouped_threads<F>(), group_tiles_max(c.rows, c.G, kTokTile) * a.tiles_n,
                        smem, a, s);
}

template <Out OT, bool kRes>
cudaError_t go_wgrad(const GroupedCall& c, cudaStream_t s) {
    WgradArgs a;
    std::memset(&a, 0, sizeof(a));
    const int kb = k_tiles<F8>(c.K);  // K: the padded tokens
    if (!code_map(&a.ta, c.a, c.M, c.K, 128) || !code_map(&a.tb, c.b, c.N, c.K, 96) ||
        !scale_map(&a.tsa, c.as, c.M, kb, 1, kSfChunkTiles) ||
        !scale_map(&a.tsb, c.bs, c.N, kb, 2, kSfChunkTiles) ||
        !chunk_map<OT>(&a.tout, c.ep.out, c.G * c.M, c.N) ||
        (kRes && !chunk_map<OT>(&a.tres, c.ep.residual, c.G * c.M, c.N)))
        return cudaErrorInvalidValue;
    a.ep = c.ep;
    a.offs = c.offs;
    a.G = c.G;
    a.rows = (int)c.rows;
    a.M = (int)c.M;
    a.N = (int)c.N;
    a.tiles_m = (int)((c.M + kPairM - 1) / kPairM);
    a.tiles_n = (int)((c.N + kPairN - 1) / kPairN);
    // Four tile rows: a group's columns are few, so both operands stay in L2 in any
    // order, and out is written in pieces of rows that lie close (8 x 14336 x 4096 fp32 of
    // 8192 tokens: 438 us; 1 row 449, 8 rows 438 .. 455, all of them 477).
    a.band = 4;
    constexpr int kOwn = 2048;
    constexpr int kOther = 4 * wgrad_slots<kRes>() * kChunkBytes + sf_slots<F8>() * kSfChunkBytes;
    static_assert((kSmemLimit - kOwn - 1024 - kOther - (int)group_table_bytes(kMaxGroups)) / kPairStageBytes >=
                      kSfBufs, "stages");
    const int table = (int)group_table_bytes(c.G);
    a.stages = (kSmemLimit - kOwn - 1024 - kOther - table) / kPairStageBytes;
    if (a.stages > kPairMaxStages) a.stages = kPairMaxStages;
    const int smem = a.stages * kPairStageBytes + kOther + table + 1024;
    return launch_pairs(k_grouped_wgrad<OT, kRes>, kOwn, pair_threads<F8>(), (int64_t)c.G * a.tiles_m * a.tiles_n, smem, a, s);
}

template <class F>
cudaError_t by_out(const GroupedCall& c, cudaStream_t s) {
    switch (c.out) {
        case In::BF16: return go<F, Out::BF16>(c, s);
        case In::F16: return go<F, Out::F16>(c, s);
        case In::F32: return go<F, Out::F32>(c, s);
    }
    return cudaErrorInvalidValue;
}

template <bool kRes>
cudaError_t wgrad_by_out(const GroupedCall& c, cudaStream_t s) {
    switch (c.out) {
        case In::BF16: return go_wgrad<Out::BF16, kRes>(c, s);
        case In::F16: return go_wgrad<Out::F16, kRes>(c, s);
        case In::F32: return go_wgrad<Out::F32, kRes>(c, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace lin

cudaError_t launch_grouped(const GroupedCall& c, cudaStream_t s) {
    if (c.wgrad) return c.ep.residual ? lin::wgrad_by_out<true>(c, s) : lin::wgrad_by_out<false>(c, s);
    return c.fmt4 ? lin::by_out<lin::F4>(c, s) : lin::by_out<lin::F8>(c, s);
}

}  // namespace fos
