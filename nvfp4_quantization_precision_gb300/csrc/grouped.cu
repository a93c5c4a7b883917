// grouped.cu -- launches of the products grouped by expert (fos_grouped.cuh).
#include <cstring>

#include "fos_grouped.cuh"
#include "fos_linear_host.cuh"

namespace fos {
namespace lin {

namespace {

template <class F, Out OT, bool kW>
cudaError_t go(const GroupedCall& c, cudaStream_t s) {
    GroupedArgs a;
    std::memset(&a, 0, sizeof(a));
    // bytes of a row of codes; of a weight gradient's columns they are the tokens
    const int64_t row_bytes = F::kGlobal ? c.K / 2 : c.K;
    const int64_t rows_a = kW ? c.M : c.rows, rows_b = kW ? c.N : c.G * c.N;
    const int64_t rows_out = kW ? c.G * c.M : c.rows;
    a.kb = k_tiles<F>(c.K);
    a.nkb = k_stages<F>(c.K);
    a.row_tiles_b = (int)((c.N + 127) / 128);
    if (!code_map(&a.ta, c.a, rows_a, row_bytes, 128) || !code_map(&a.tb, c.b, rows_b, row_bytes, 96) ||
        (!kW && !code_map(&a.ta32, c.a, rows_a, row_bytes, 32)) ||
        (kW && !scale_map(&a.tsa, c.as, rows_a, a.kb, 1, kSfChunkTiles)) ||
        !scale_map(&a.tsb, c.bs, kW ? rows_b : (int64_t)c.G * a.row_tiles_b * 128, a.kb, 2, kSfChunkTiles) ||
        !chunk_map<OT>(&a.tout, c.ep.out, rows_out, c.N) ||
        (c.ep.residual && !chunk_map<OT>(&a.tres, c.ep.residual, rows_out, c.N)) ||
        (c.ep.pre && !chunk_map<OT>(&a.tpre, c.ep.pre, rows_out, c.N)))
        return cudaErrorInvalidValue;
    a.ep = c.ep;
    a.sa = c.as;
    a.sa_pitch = F::kGlobal ? c.K / 16 : c.K / 32;
    a.sa_wide = a.sa_pitch % 16 == 0;
    a.offs = c.offs;
    a.G = c.G;
    a.rows = (int)c.rows;
    a.M = (int)c.M;
    a.N = (int)c.N;
    a.tiles_m = (int)((c.M + kPairM - 1) / kPairM);
    a.tiles_n = (int)((c.N + kPairN - 1) / kPairN);
    // Bands of tile rows whose rows of a take at most 30 MB, a quarter of L2 (pair_go());
    // of a weight gradient's columns a group has its share.
    const int64_t band_bytes = kPairM * (kW ? row_bytes / c.G + 1 : row_bytes);
    const int64_t fit = 30000000 / band_bytes;
    a.band = (int)(fit < 1 ? 1 : fit > 4096 ? 4096 : fit);
    a.bufs = c.ep.pre ? 4 : 2;
    const int table = (int)group_table_bytes(c.G);
    const int other = 4 * a.bufs * kChunkBytes + sf_slots<F>() * kSfChunkBytes + 4 * kPairN * 4 + table;
    static_assert((kSmemLimit - 2048 - 16 * kChunkBytes - kSfMaxSlots * kSfChunkBytes - 16 * kPairN -
                   (int)group_table_bytes(kMaxGroups)) / kPairStageBytes >= kSfBufs, "stages");
    a.stages = (kSmemLimit - 2048 - other) / kPairStageBytes;
    if (a.stages > kPairMaxStages) a.stages = kPairMaxStages;
    const int smem = a.stages * kPairStageBytes + other + 1024;
    auto k = k_grouped<F, OT, kW>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), (size_t)kSmemLimit - 1024);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (kW ? (int64_t)c.G * a.tiles_m : group_tiles_max(c.rows, c.G, 8)) * a.tiles_n;
    int64_t clusters = resident_clusters(k, pair_threads<F>(), smem, 2);
    if (clusters > tiles) clusters = tiles;
    return launch_clusters(k, (int)clusters, 2, pair_threads<F>(), smem, a, s);
}

template <class F, bool kW>
cudaError_t by_out(const GroupedCall& c, cudaStream_t s) {
    switch (c.out) {
        case In::BF16: return go<F, Out::BF16, kW>(c, s);
        case In::F16: return go<F, Out::F16, kW>(c, s);
        case In::F32: return go<F, Out::F32, kW>(c, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace lin

cudaError_t launch_grouped(const GroupedCall& c, cudaStream_t s) {
    if (c.wgrad) return lin::by_out<lin::F8, true>(c, s);
    return c.fmt4 ? lin::by_out<lin::F4, false>(c, s) : lin::by_out<lin::F8, false>(c, s);
}

}  // namespace fos
