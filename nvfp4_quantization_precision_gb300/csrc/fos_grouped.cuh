// fos_grouped.cuh -- products of rows packed by group (expert) with the groups'
// own weights, and the weights' gradients, on pairs of SMs (tcgen05
// cta_group::2, M = 256).
//
//   kW false  out[m] = act(a[m] . b[e]^T + bias[e]) + residual[m], e the group of
//             row m: tiles of 256 rows of one group x 192 weight rows; the groups'
//             rows are ragged, every tile's K is K.
//   kW true   out[e] = a[:, e] . b[:, e]^T + residual[e], a and b column-wise 8-bit
//             forms whose columns are the tokens, each group's part a whole number
//             of 128: tiles of 256 x 192 of out[e], K the group's columns (none:
//             the product is 0).
//
// The host knows neither the groups' sizes nor the number of tiles: every CTA reads
// the ends (fos_groups.cuh) and walks tiles t, t + pairs, ... of the groups one
// after the other, each role for itself.  Roles, rings, tensor memory and the
// epilogue's chunks are those of k_linear_pair; what differs:
//   rows of a   a tile's last rows may be another group's: boxes of 32 rows fetch
//               what the group has (with one row an expert, 4 KB a stage instead
//               of 16 per SM: the weights are then all that streams), and the rest of
//               the stage keeps what it held.  Those rows of the accumulator are
//               nobody's: a row of the product depends on its own row of a alone.
//   scales of a are plain, [rows, K / 16 or K / 32] as the quantizers write packed rows:
//               a tile starts at any row, and a 128-row tile of scales could not
//               start there.  Warp 10 copies 16 bytes (four scale tiles along K) a
//               row by cp.async, and the lanes that hold rows l, 32 + l, 64 + l, 96 +
//               l read them as they are.
//   rows of out a chunk of 32 rows that the group fills leaves by TMA; one that it
//               ends in is copied row by row.
#pragma once

#include "fos_groups.cuh"
#include "fos_linear_pair.cuh"

namespace fos {

// One grouped product or weight gradient, as the host passes it to the launcher.
struct GroupedCall {
    const uint8_t *a, *as, *b, *bs;  // codes and scales
    const int32_t* offs;
    int G;
    int64_t rows;                    // packed rows
    int64_t M, N, K;                 // rows of a tile grid (weight gradient), columns of out, K
    Epilogue ep;
    In out;
    bool fmt4, wgrad;
};

namespace lin {

struct GroupedArgs {
    CUtensorMap ta;    // a codes, box 128 bytes x 128 rows
    CUtensorMap ta32;  // the same, 32 rows (kW false)
    CUtensorMap tb;    // b codes, box 128 bytes x 96 rows, the groups' weights below one another
    CUtensorMap tsa;   // kW: a's tiled scales, box 1 x 4 x 512
    CUtensorMap tsb;   // b's tiled scales, box 2 x 4 x 512
    CUtensorMap tout;  // out, residual, pre: box 128 bytes x 32 rows
    CUtensorMap tres;
    CUtensorMap tpre;
    Epilogue ep;
    const uint8_t* sa;     // plain scales of a
    int64_t sa_pitch;      // bytes of a row of them
    int sa_wide;           // rows of them are whole 16-byte pieces
    const int32_t* offs;
    int G;
    int rows;              // packed rows
    int M;                 // kW: rows of out[e]
    int N;                 // columns of out
    int tiles_m;           // kW: row tiles of out[e]
    int tiles_n;
    int band;
    int kb, nkb;           // kW false: scale tiles and stages along K
    int row_tiles_b;       // kW false: scale row tiles of one group's weights
    int stages, bufs;
};

// One tile of the walk.
struct GroupedTile {
    int g;
    int32_t m0, m_end;   // rows of a (and of out, from out_row) and where they end
    int32_t n0;
    int32_t k0, nkb;     // first stage of a's columns, stages
    int32_t out_row;     // out's row of a's row 0
};

template <bool kW>
__device__ __forceinline__ int grouped_tiles(const GroupedArgs& a, const Group* t) {
    return (kW ? a.G * a.tiles_m : t[a.G].tile) * a.tiles_n;
}
// Within a group, bands of a.band tile rows, down the rows first (pair_tile()).
template <bool kW>
__device__ __forceinline__ void grouped_tile(const GroupedArgs& a, const Group* t, int tile,
                                             GroupedTile& w) {
    const int q = tile / a.tiles_n;
    const int g = kW ? q / a.tiles_m : group_of(t, a.G, q, w.g);
    const int base = kW ? g * a.tiles_m : t[g].tile;
    const int all = kW ? a.tiles_m : t[g + 1].tile - base;
    const int r0 = tile - base * a.tiles_n;
    const int per_band = a.band * a.tiles_n;
    const int band = r0 / per_band, r = r0 - band * per_band;
    const int rows = min(a.band, all - band * a.band);
    const int col = r / rows;
    const int m = (band * a.band + r - col * rows) * kPairM;
    w.g = g;
    w.n0 = col * kPairN;
    if constexpr (kW) {
        w.m0 = m;
        w.m_end = a.M;
        w.k0 = t[g].tile;
        w.nkb = t[g + 1].tile - w.k0;
        w.out_row = g * a.M;
    } else {
        w.m0 = t[g].row + m;
        w.m_end = t[g + 1].row;
        w.k0 = 0;
        w.nkb = a.nkb;
        w.out_row = 0;
    }
}
// Rows of the tile that CTA `rank` of the pair has.
__device__ __forceinline__ int rank_rows(const GroupedTile& w, int rank) {
    return max(0, min(128, w.m_end - w.m0 - 128 * rank));
}
// Boxes of 32 rows that fetch them (more than three: one box of 128).
__device__ __forceinline__ int a_boxes(int rows) { return (rows + 31) >> 5; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// This thread's arrival at `bar` once its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The first `rows` rows of a 32-row chunk to `dst` [.., N] at (row, col): eight
// lanes a row, as far as the columns go.
template <Out OT>
__device__ __forceinline__ void copy_rows(uint32_t buf, void* dst, int64_t row, int col, int N,
                                          int rows, int lane) {
    constexpr int kElt = OT == Out::F32 ? 4 : 2;
    const int piece = lane & 7, c = col + piece * (16 / kElt);
    if (c >= N) return;
    for (int r = lane >> 3; r < rows; r += 4) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(buf + r * 128 + ((piece ^ (r & 7)) << 4)) : "memory");
        st128(static_cast<char*>(dst) + ((row + r) * (int64_t)N + c) * kElt, w);
    }
}

template <class F, Out OT, bool kW>
__global__ void __launch_bounds__(pair_threads<F>(), 1) k_grouped(const __grid_constant__ GroupedArgs a) {
    extern __shared__ __align__(1024) unsigned char s_raw[];
    __shared__ PairShared sh;
    unsigned char* base = s_raw + ((1024u - (smem_u32(s_raw) & 1023u)) & 1023u);
    const int ns = a.stages;
    constexpr int kSfSlots = sf_slots<F>();
    unsigned char* sA = base;
    unsigned char* sB = sA + ns * kPairABytes;
    unsigned char* sC = sB + ns * kPairBBytes;          // epilogue chunks
    unsigned char* sS = sC + 4 * a.bufs * kChunkBytes;  // scale chunks: a, then b's two row tiles
    float* sBias = reinterpret_cast<float*>(sS + kSfSlots * kSfChunkBytes);
    Group* groups = reinterpret_cast<Group*>(sBias + 4 * kPairN);
    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int rank = (int)uniform(cluster_rank());
    const int first = (int)(blockIdx.x >> 1), step = (int)(gridDim.x >> 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < ns; ++s) {
            bar_init(&sh.full[s], chunk_is_stage<F>() ? 9 : 1);
            bar_init(&sh.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(&sh.acc_full[b], 1);
            bar_init(&sh.acc_empty[b], 8);
        }
        for (int b = 0; b < kSfSlots; ++b) {
            bar_init(&sh.sf_full[b], kW ? 1 : 33);  // and each lane's copies of a's scales
            bar_init(&sh.sf_empty[b], 4);
        }
        for (int b = 0; b < kSfBufs; ++b) {
            bar_init(&sh.sf_ready[b], 8);
            bar_init(&sh.sf_free[b], 1);
        }
        for (int w = 0; w < 4; ++w)
            for (int b = 0; b < 2; ++b) bar_init(&sh.res_full[w][b], 1);
        bar_init(&sh.done, 1);
        sh.fail = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    chain_wait();
    chain_release();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh.tmem)), "r"(kAllColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else if (warp == 2) {
        group_table<kW ? 7 : 8>(groups, a.offs, a.G, a.rows, lane);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are set up
    tc_fence_after();
    const uint32_t tmem = uniform(sh.tmem);
    const int tiles = grouped_tiles<kW>(a, groups);
    GroupedTile w;
    w.g = 0;
    bool bad = false;
    if (warp == 0) {
        const bool elected = elect_lane();
        const uint32_t full0 = map_rank(smem_u32(&sh.full[0]), 0);
        Ring r;
        uint32_t g = 0;
        for (int t = first; t < tiles && !bad; t += step) {
            grouped_tile<kW>(a, groups, t, w);
            const int32_t am = w.m0 + 128 * rank;
            const int32_t bn = (kW ? 0 : w.g * a.N) + w.n0 + 96 * rank;
            // the pair's rows, in boxes; past the last row a weight gradient's boxes read zeros
            const int mine = kW ? 4 : a_boxes(rank_rows(w, rank));
            const int both = kW ? 8 : a_boxes(rank_rows(w, 0)) + a_boxes(rank_rows(w, 1));
            const uint32_t bytes = (uint32_t)(2 * kPairBBytes + both * (kPairABytes / 4));
            for (int i = 0; i < w.nkb; ++i) {
                const int s = r.slot;
                if (g >= (uint32_t)ns && !warp_wait<Sync::CLUSTER>(&sh.empty[s], r.parity ^ 1u)) {
                    bad = true;
                    break;
                }
                const uint32_t bar = full0 + 8 * s;
                const int32_t x = (w.k0 + i) * kRowBytes;
                unsigned char *pa = sA + s * kPairABytes, *pb = sB + s * kPairBBytes;
                if (elected) {
                    if (rank == 0) mbar_expect_tx(&sh.full[s], bytes);
                    if (mine == 4) {
                        pair_load_2d(pa, &a.ta, x, am, bar);
                    } else {
                        for (int j = 0; j < mine; ++j)
                            pair_load_2d(pa + j * (kPairABytes / 4), &a.ta32, x, am + 32 * j, bar);
                    }
                    pair_load_2d(pb, &a.tb, x, bn, bar);
                }
                __syncwarp();
                ++g;
                r.next(ns);
            }
        }
        // every copy issued has landed (and been read) before the CTA leaves:
        // the stages' last uses, by the barriers this CTA has
        for (int k = 0; k < ns && (uint32_t)k < g; ++k) {
            int s = r.slot - 1 - k;
            uint32_t p = r.parity;
            if (s < 0) {
                s += ns;
                p ^= 1u;
            }
            if (!warp_wait<Sync::CLUSTER>(&sh.empty[s], p)) bad = true;
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const bool elected = elect_lane();
            Ring r, f;          // stages; scale buffers
            bool here = false;  // the next stage is known to be full
            int j = 0;          // accumulators used
            for (int t = first; t < tiles && !bad; t += step) {
                grouped_tile<kW>(a, groups, t, w);
                if (kW && w.nkb == 0) continue;  // no accumulator: the epilogue takes zeros
                const int ab = j & 1;
                if (j >= 2 && !warp_wait<Sync::TENSOR>(&sh.acc_empty[ab], (uint32_t)((j >> 1) - 1) & 1)) {
                    bad = true;
                    break;
                }
                ++j;
                const uint32_t acc = tmem + (uint32_t)(ab * kPairN);
                const int kb = kW ? w.nkb : a.kb;
                for (int i = 0; i < w.nkb; ++i) {
                    const int s = r.slot, in_chunk = i % chunk_stages<F>();
                    if ((!chunk_is_stage<F>() && in_chunk == 0 &&
                         !warp_wait<Sync::TENSOR>(&sh.sf_ready[f.slot], f.parity)) ||
                        (!warp_agrees(here) && !warp_wait<Sync::CLUSTER>(&sh.full[s], r.parity))) {
                        bad = true;
                        break;
                    }
                    r.next(ns);
                    tc_fence_after();
                    const int nk = min(F::kSfTiles, kb - F::kSfTiles * i);
                    const uint32_t a0 = desc_lo(smem_u32(sA) + s * kPairABytes);
                    const uint32_t b0 = desc_lo(smem_u32(sB) + s * kPairBBytes);
                    const uint32_t sf = tmem + kPairSfCol + f.slot * kSfCols;
                    const bool last = in_chunk == chunk_stages<F>() - 1 || i + 1 == w.nkb;
                    if (elected) {
                        pair_stage<F>(acc, a0, b0, sf + 4 * in_chunk, sf + 16 + 6 * in_chunk, nk, i > 0);
                        pair_commit(&sh.empty[s]);
                        if (!chunk_is_stage<F>() && last) pair_commit(&sh.sf_free[f.slot]);
                    }
                    here = mbar_ask<Sync::CLUSTER>(&sh.full[r.slot], r.parity);
                    __syncwarp();
                    if (last) f.next(kSfBufs);
                }
                if (!bad && elected) pair_commit(&sh.acc_full[ab]);
                __syncwarp();
            }
            if (elected) pair_commit(&sh.done);
            __syncwarp();
        }
    } else if (warp == 10) {
        const bool elected = elect_lane();
        Ring f;
        uint32_t chunks = 0;
        for (int t = first; t < tiles && !bad; t += step) {
            grouped_tile<kW>(a, groups, t, w);
            const int32_t ra = (w.m0 + 128 * rank) >> 7;
            const int32_t rb = (kW ? 0 : w.g * a.row_tiles_b) + (w.n0 >> 7);
            const int mine = rank_rows(w, rank);
            const uint8_t* src = kW ? nullptr : a.sa + (int64_t)(w.m0 + 128 * rank) * a.sa_pitch;
            const int kb = kW ? w.nkb : a.kb;
            for (int k = 0; k < kb; k += kSfChunkTiles) {
                if (chunks >= (uint32_t)kSfSlots && !warp_wait(&sh.sf_empty[f.slot], f.parity ^ 1u)) {
                    bad = true;
                    break;
                }
                unsigned char* ps = sS + f.slot * kSfChunkBytes;
                uint64_t* bar = &sh.sf_full[f.slot];
                if (elected) {
                    mbar_expect_tx(bar, (uint32_t)(kW ? kSfChunkBytes : kSfChunkBytes - kSfChunkA));
                    if (kW) sf_load_3d(ps, &a.tsa, w.k0 + k, ra, bar);
                    sf_load_3d(ps + kSfChunkA, &a.tsb, w.k0 + k, rb, bar);
                }
                __syncwarp();
                if constexpr (!kW) {
                    for (int r = lane; r < mine; r += 32) {
                        const uint8_t* p = src + r * a.sa_pitch + 4 * k;
                        const uint32_t d = smem_u32(ps) + 16 * r;
                        if (a.sa_wide) {
                            cp_async16(d, p);
                        } else {
                            for (int j = 0; j < min(kSfChunkTiles, kb - k); ++j) cp_async4(d + 4 * j, p + 4 * j);
                        }
                    }
                    cp_async_arrive(bar);
                    __syncwarp();
                }
                ++chunks;
                f.next(kSfSlots);
            }
        }
        // the chunks' last uses have landed and been read
        for (int k = 0; k < kSfSlots && (uint32_t)k < chunks; ++k) {
            int sl = f.slot - 1 - k;
            uint32_t p = f.parity;
            if (sl < 0) {
                sl += kSfSlots;
                p ^= 1u;
            }
            if (!warp_wait(&sh.sf_empty[sl], p)) bad = true;
        }
    } else if (warp < 6 || warp > 10) {
        // scales: lane l of quadrant q writes a's of rows l, 32 + l, 64 + l, 96 + l to
        // columns 4 kk ..., of b's eight words (two row tiles) the six of the tile's
        // 192 rows to columns 16 + 6 kk ...
        const int q = warp & 3;
        const uint32_t lane_base = tmem + kPairSfCol + ((uint32_t)(32 * q) << 16);
        const uint32_t full0 = map_rank(smem_u32(&sh.full[0]), 0);
        const uint32_t ready0 = map_rank(smem_u32(&sh.sf_ready[0]), 0);
        Ring f, d;          // shared-memory slots; tensor-memory buffers
        Ring r, u;          // chunk_is_stage: its stage; the one whose buffer it takes over
        const uint32_t mine = warp < 6 ? 0u : 1u;  // the group of scale warps
        uint32_t chunks = 0;
        for (int t = first; t < tiles && !bad; t += step) {
            grouped_tile<kW>(a, groups, t, w);
            const bool half = (w.n0 & 127) != 0;  // b starts half-way into a scale tile
            for (int i = 0; i < w.nkb; i += chunk_stages<F>()) {
                if (chunks % sf_groups<F>() != mine) {
                    if (chunks >= (uint32_t)kSfBufs) u.next(ns);
                    ++chunks;
                    r.next(ns);
                    f.next(kSfSlots);
                    d.next(kSfBufs);
                    continue;
                }
                if (!warp_wait(&sh.sf_full[f.slot], f.parity)) {
                    bad = true;
                    break;
                }
                const unsigned char* ps = sS + f.slot * kSfChunkBytes + 16 * lane;
                uint32_t va[16], vb[24];
#pragma unroll
                for (int kk = 0; kk < kSfChunkTiles; ++kk) {
                    // kW: tile kk, rows l ... in its words; else rows 32 kk + l, tiles in the words
                    const uint4 x = *reinterpret_cast<const uint4*>(ps + kk * kSfTileBytes);
                    const uint4 y = *reinterpret_cast<const uint4*>(ps + kSfChunkA + kk * kSfTileBytes);
                    const uint4 z = *reinterpret_cast<const uint4*>(ps + 2 * kSfChunkA + kk * kSfTileBytes);
                    constexpr int kA = kW ? 1 : 4;
                    const int a0 = kW ? 4 * kk : kk;
                    va[a0] = x.x; va[a0 + kA] = x.y; va[a0 + 2 * kA] = x.z; va[a0 + 3 * kA] = x.w;
                    vb[6 * kk] = half ? y.z : y.x;
                    vb[6 * kk + 1] = half ? y.w : y.y;
                    vb[6 * kk + 2] = half ? z.x : y.z;
                    vb[6 * kk + 3] = half ? z.y : y.w;
                    vb[6 * kk + 4] = half ? z.z : z.x;
                    vb[6 * kk + 5] = half ? z.w : z.y;
                }
                if (chunks >= (uint32_t)kSfBufs) {
                    // the MMAs that read this buffer are done
                    if (chunk_is_stage<F>() ? !warp_wait<Sync::TENSOR>(&sh.empty[u.slot], u.parity)
                                            : !warp_wait<Sync::TENSOR>(&sh.sf_free[d.slot], d.parity ^ 1u)) {
                        bad = true;
                        break;
                    }
                    u.next(ns);
                }
                tc_fence_after();
                const uint32_t col = lane_base + d.slot * kSfCols;
                mma::tmem_st_x16(col, va);
                mma::tmem_st_x16(col + 16, reinterpret_cast<uint32_t(&)[16]>(vb));
                tmem_st_x8(col + 32, vb + 16);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    cluster_arrive(chunk_is_stage<F>() ? full0 + 8 * r.slot : ready0 + 8 * d.slot);
                    // The slot is free once its values are in tensor memory: freed before
                    // the stores that use them, its last loads were found moved behind the
                    // arrival and took the slot's next chunk.
                    bar_arrive(&sh.sf_empty[f.slot]);
                }
                r.next(ns);
                ++chunks;
                f.next(kSfSlots);
                d.next(kSfBufs);
            }
        }
    } else {
        const int q = warp & 3, e = warp - 6;
        constexpr int kElt = OT == Out::F32 ? 4 : 2;
        constexpr int kCols = 128 / kElt;               // columns of a chunk
        constexpr int kChunks = kPairN / kCols;         // chunks of a tile
        const bool pre = !kW && a.ep.pre != nullptr, res = a.ep.residual != nullptr;
        const bool has_bias = !kW && a.ep.bias != nullptr;
        // two slots of a buffer for out (and the residual) and, with pre, one for it
        const int slot_bytes = (pre ? 2 : 1) * kChunkBytes;
        unsigned char* bufs = sC + e * 2 * slot_bytes;
        float* s_bias = sBias + e * kPairN;
        int c = 0, j = 0;  // chunks of this warp, accumulators used
        for (int t = first; t < tiles; t += step) {
            grouped_tile<kW>(a, groups, t, w);
            const int32_t mw = w.m0 + 128 * rank + 32 * q;           // first row of this warp
            const int live = max(0, min(32, w.m_end - mw));          // rows of the group
            const int32_t orow = w.out_row + mw;
            auto fetch = [&](int k) {                                // chunk k's residual (one lane)
                uint64_t* bar = &sh.res_full[e][c & 1];
                mbar_expect_tx(bar, kChunkBytes);
                tma_load_2d(bufs + (c & 1) * slot_bytes, &a.tres, w.n0 + k * kCols, orow, bar);
            };
            if (res && live > 0 && lane == 0) fetch(0);
            float ga = 1.0f, gb = 1.0f;
            if constexpr (F::kGlobal) {
                gb = fdiv(1.0f, global_scale(a.ep.b_amax[w.g], a.ep.six_bound));
                if (lane < live)
                    ga = fdiv(1.0f, global_scale(a.ep.a_amax[a.ep.a_row ? mw + lane : w.g], a.ep.six_bound));
            }
            if (has_bias && live > 0) {
                float bias[kPairN / 32];
                Epilogue ep = a.ep;
                ep.bias = static_cast<const char*>(a.ep.bias) + (int64_t)w.g * a.N * (a.ep.bias32 ? 4 : kElt);
                load_bias<OT>(ep, w.n0, a.N, lane, bias);
#pragma unroll
                for (int i = 0; i < kPairN / 32; ++i) s_bias[32 * i + lane] = bias[i];
            }
            const bool sum = !kW || w.nkb > 0;  // there is a product
            const int ab = j & 1;
            if (sum) {
                if (!bad && !warp_wait<Sync::TENSOR>(&sh.acc_full[ab], (uint32_t)(j >> 1) & 1)) bad = true;
                ++j;
            }
            __syncwarp();
            tc_fence_after();
            if (live == 0) {
                if (sum) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) cluster_arrive(map_rank(smem_u32(&sh.acc_empty[ab]), 0));
                }
                continue;
            }
            for (int k = 0; k < kChunks; ++k, ++c) {
                const uint32_t buf = smem_u32(bufs + (c & 1) * slot_bytes);
                if (res && !bad && !warp_wait(&sh.res_full[e][c & 1], (uint32_t)(c >> 1) & 1)) bad = true;
                __syncwarp();
#pragma unroll
                for (int h = 0; h < kCols / 32; ++h) {
                    const int32_t col = k * kCols + 32 * h;
                    uint32_t u[32];
                    if (sum) {
                        tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(ab * kPairN + col), u);
                        if (col + 32 == kPairN) {  // this warp has read the accumulator
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) cluster_arrive(map_rank(smem_u32(&sh.acc_empty[ab]), 0));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) u[i] = 0u;
                    }
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        v[i] = __uint_as_float(u[i]);
                        if constexpr (F::kGlobal) v[i] = fmul(fmul(v[i], ga), gb);
                    }
                    if (has_bias) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 b4 = *reinterpret_cast<const float4*>(s_bias + col + 4 * i);
                            v[4 * i] = fadd(v[4 * i], b4.x);
                            v[4 * i + 1] = fadd(v[4 * i + 1], b4.y);
                            v[4 * i + 2] = fadd(v[4 * i + 2], b4.z);
                            v[4 * i + 3] = fadd(v[4 * i + 3], b4.w);
                        }
                    }
                    constexpr int kPieces = 32 * kElt / 16;
                    if (pre) put_pieces<OT>(buf + kChunkBytes + lane * 128, lane, kPieces * h, v);
                    if constexpr (!kW) act_apply<OT>(a.ep.act, v);
                    if (res) add_pieces<OT>(buf + lane * 128, lane, kPieces * h, v);
                    put_pieces<OT>(buf + lane * 128, lane, kPieces * h, v);
                }
                const int32_t n = w.n0 + k * kCols;
                if (live < 32) {  // the rows below are another group's
                    __syncwarp();
                    copy_rows<OT>(buf, a.ep.out, orow, n, a.N, live, lane);
                    if (pre) copy_rows<OT>(buf + kChunkBytes, a.ep.pre, orow, n, a.N, live, lane);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    if (live == 32) {
                        store_chunk(&a.tout, n, orow, buf);
                        if (pre) store_chunk(&a.tpre, n, orow, buf + kChunkBytes);
                    }
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    // the chunk before this one has left its slot, which the
                    // next one is fetched into and written to
                    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                    if (res && k + 1 < kChunks) {
                        uint64_t* bar = &sh.res_full[e][(c + 1) & 1];
                        mbar_expect_tx(bar, kChunkBytes);
                        tma_load_2d(bufs + ((c + 1) & 1) * slot_bytes, &a.tres, n + kCols, orow, bar);
                    }
                }
            }
            __syncwarp();  // the biases are read before the next tile's replace them
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    // every MMA issued has completed before the tensor memory is freed
    if (warp == 1 && !warp_wait<Sync::TENSOR>(&sh.done, 0)) bad = true;
    if (bad) sh.fail = 1;
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other may touch its memory
    if (sh.fail && threadIdx.x == 0 && first < tiles) {
        grouped_tile<kW>(a, groups, first, w);
        store_out<OT>(a.ep.out, (int64_t)(w.out_row + w.m0) * a.N + w.n0, __int_as_float(0x7FC00000));
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kAllColumns) : "memory");
    }
}

}  // namespace lin
}  // namespace fos
