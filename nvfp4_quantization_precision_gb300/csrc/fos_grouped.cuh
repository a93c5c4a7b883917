// fos_grouped.cuh -- products of rows packed by group (expert) with the groups'
// own weights, and the weights' gradients, on pairs of SMs (tcgen05 cta_group::2, M =
// 256).  The host knows neither the groups' sizes nor the number of tiles: every CTA
// reads the ends (fos_groups.cuh) and walks tiles t, t + pairs, ... of the groups one
// after the other, each role for itself.  Roles, rings, tensor memory and the waits
// are those of k_linear_pair.
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
    int64_t M, N, K;                 // rows of out[e] (weight gradient), columns of out, K
    Epilogue ep;
    In out;
    bool fmt4, wgrad;
};

namespace lin {

// The pair's halves of a stage: 128 rows of the first operand, up to 96 of the second.
static_assert(kPairABytes == 128 * kRowBytes && kPairBBytes == 96 * kRowBytes, "stage");

// ------------------------------------------------------------------ out = act(a . b[e]^T ...)
// k_grouped: the weights are the MMA's 256 rows and a group's rows (tokens) its
// columns, as in k_linear_rows, so that a tile that the group ends in costs what it has:
// tiles of 256 weight rows x 192 tokens, the last one of a group as many as it
// needs, rounded up to 32 (a group's tokens in even parts: prefill of 16384 tokens over
// 63 experts 140 us instead of 127).  (With tokens as the 256 rows, groups of 255 rows on average
// fill 60 % of their tiles: 16084 x 2048 x 7168 NVFP4 over 63 groups 182 us.)
// CTA r of a pair holds weight rows 128 r .. + 127 of the tile and its half of the
// tokens; each CTA's tensor memory has the products of its weight rows and all of
// the tokens.  What differs from k_linear_pair besides:
//   tokens     a tile starts at any row: a last tile's are fetched by boxes of 16 rows,
//              which may hold another group's behind the end: their columns of the
//              product are nobody's
//   scales     of the weights are tiled, of the tokens plain, [rows, K / 16 or K / 32],
//              as the quantizers write packed rows (a 128-row tile of scales could not
//              start at any row): warp 10 copies 16 bytes (four scale tiles along K) a
//              token by cp.async, and the lanes that hold tokens l, 32 + l, ... read them
//              as they are
//   epilogue   a lane has one weight row: its 32 neighbours' results of a token are 64
//              or 128 contiguous bytes of out, stored as they are, without a way through
//              shared memory; by eight warps, two a quadrant, which take every other 16
//              tokens (1003 tokens x 1040 x 640 with everything, one tile a pair: 13.1 us
//              with four, 12.2 with eight).  The residual comes by TMA, kResSlots - 1
//              chunks ahead.  With K of some hundreds the epilogue is what a tile takes:
//              two warps a scheduler, some 190 instructions a chunk of 16 tokens (tokens
//              stored without a predicate where a chunk is full: up to 3 % slower)

constexpr int kTokTile = 192;                    // tokens of a tile
constexpr int kTokStep = 32;                     // an MMA's columns come in steps of these
constexpr int kTokBox = 16;                      // tokens of a small box
constexpr int kTokSfBytes = kTokTile * 16;       // a chunk of their scales
constexpr int kGrpSfBytes = kSfChunkA + kTokSfBytes;
// Chunks of scales in shared memory: of NVFP4, whose chunk is a stage, two are held by
// the groups of scale warps while they wait for a buffer in tensor memory, and the
// others have to cover the copies' latency.
template <class F> constexpr int grp_slots() { return F::kGlobal ? 8 : 3; }

// Four more warps than k_linear_pair: the second half of the epilogue.
template <class F> constexpr int grouped_threads() { return pair_threads<F>() + 128; }
constexpr int kEpiTok = 16;                      // tokens of a chunk of the epilogue
// The residual's chunks of a warp of the epilogue in shared memory: kEpiTok rows of 32 values.
template <Out OT> constexpr int grp_res_bytes() { return kEpiTok * 32 * (OT == Out::F32 ? 4 : 2); }
template <Out OT> constexpr int grp_res_slots() { return OT == Out::F32 ? 3 : 4; }

struct __align__(8) GroupedShared {
    uint64_t full[kPairMaxStages], empty[kPairMaxStages], acc_full[2], acc_empty[2], done;
    uint64_t sf_full[8], sf_empty[8], sf_ready[kSfBufs], sf_free[kSfBufs];
    uint32_t tmem;
    int fail;
};

struct GroupedArgs {
    CUtensorMap tw;    // weights' codes, box 128 bytes x 128 rows, the groups' below one another
    CUtensorMap tt;    // tokens' codes, box 128 bytes x 96 rows
    CUtensorMap tt16;  // the same, 16 rows
    CUtensorMap tsw;   // weights' tiled scales, box 1 x 4 x 512
    CUtensorMap tst;   // ts_wide: the tokens' plain scales, box 16 bytes x 192 rows
    CUtensorMap tst32; // the same, 32 rows
    CUtensorMap tres;  // residual [rows, N]: box 32 x kEpiTok
    Epilogue ep;
    const uint8_t* ts;     // plain scales of the tokens
    int64_t ts_pitch;      // bytes of a row of them
    int ts_wide;           // rows of them are whole 16-byte pieces: by TMA
    const int32_t* offs;
    int G;
    int rows;              // packed rows
    int N;                 // weight rows of a group
    int tiles_n;
    int band;              // token tiles of a band of the tile order
    int kb, nkb;           // scale tiles and stages along K
    int row_tiles;         // scale row tiles of a group's weights
    int stages;
    int res_area;          // bytes of the residual's chunks of all warps (none without one)
};

// One tile of the walk.
struct GroupedTile {
    int g;
    int32_t t0, live;  // first token, tokens of the group in it
    int32_t cols;      // the same, rounded up to kTokStep
    int32_t n0;
};

// Token tiles of a band: their rows take at most 30 MB, a quarter of L2 (pair_go()), and
// they are no more than a group can have.  The latter keeps a band times the tiles of
// the weight rows below the number of all tiles, which fits 32 bits for every size that
// the calls take (rows x N up to 2^40, G x N below 2^31), and so grouped_tile()'s products.
inline int token_band(int64_t rows, int64_t row_bytes) {
    const int64_t fit = 30000000 / (kTokTile * row_bytes), all = (rows + kTokTile - 1) / kTokTile;
    return (int)(fit < 1 ? 1 : fit < all ? fit : all);
}

// Within a group, bands of a.band token tiles, down the tokens first (pair_tile()).
__host__ __device__ __forceinline__ void grouped_tile(const GroupedArgs& a, const Group* t, int tile,
                                             GroupedTile& w) {
    const int g = group_of(t, a.G, tile / a.tiles_n, w.g);
    const int all = t[g + 1].tile - t[g].tile;
    const int r0 = tile - t[g].tile * a.tiles_n;
    const int per_band = a.band * a.tiles_n;
    const int band = r0 / per_band, r = r0 - band * per_band;
    const int rows = min(a.band, all - band * a.band);
    const int col = r / rows;
    w.g = g;
    w.t0 = t[g].row + (band * a.band + r - col * rows) * kTokTile;
    w.live = min(kTokTile, t[g + 1].row - w.t0);
    w.cols = (w.live + kTokStep - 1) / kTokStep * kTokStep;
    w.n0 = col * kPairM;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// This thread's arrival at `bar` once its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The MMAs of a stage (one lane) of a tile whose instruction descriptor is `id`: nk
// scale tiles of it exist (F4).
template <class F>
__device__ __forceinline__ void grouped_stage(uint32_t acc, uint32_t a0, uint32_t b0, uint32_t id,
                                              uint32_t sfa, uint32_t sfb, int nk, uint32_t more) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
        if (F::kGlobal && kk >= nk) break;
        mma_issue<F, 2>(acc, a0 + 2 * kk, b0 + 2 * kk,
                        F::kGlobal ? id : id | ((uint32_t)kk << 4) | ((uint32_t)kk << 29),
                        F::kGlobal ? sfa + 4 * kk : sfa, F::kGlobal ? sfb + 6 * kk : sfb,
                        kk == 0 ? more : 1u);
    }
}

__device__ __forceinline__ void prefetch_chunk(const CUtensorMap* map, int32_t x, int32_t y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y) : "memory");
}

// Values of a lane's column n to rows 0 .. of `p` (at row 0, column n) below `rows`.
template <Out OT>
__device__ __forceinline__ void store_column(void* p, int64_t N, const float (&v)[kEpiTok], int rows) {
    if constexpr (OT == Out::F32) {
#pragma unroll
        for (int i = 0; i < kEpiTok; ++i)
            if (i < rows) st32(static_cast<float*>(p) + i * N, __float_as_uint(v[i]));
    } else {
#pragma unroll
        for (int i = 0; i < kEpiTok; i += 2) {
            const uint32_t w = out_pair<OT>(pk(v[i], v[i + 1]));
            if (i < rows) st16(static_cast<unsigned short*>(p) + i * N, w);
            if (i + 1 < rows) st16(static_cast<unsigned short*>(p) + (i + 1) * N, w >> 16);
        }
    }
}

template <class F, Out OT>
__global__ void __launch_bounds__(grouped_threads<F>(), 1) k_grouped(const __grid_constant__ GroupedArgs a) {
    extern __shared__ __align__(1024) unsigned char s_raw[];
    __shared__ GroupedShared sh;
    __shared__ __align__(16) float s_ga[F::kGlobal ? 8 : 1][kTokTile];  // the tokens' decode scales
    constexpr int kResSlots = grp_res_slots<OT>(), kResBytes = grp_res_bytes<OT>();
    __shared__ __align__(8) uint64_t s_res[8][kResSlots];  // the residual's chunks are here
    unsigned char* base = s_raw + ((1024u - (smem_u32(s_raw) & 1023u)) & 1023u);
    const int ns = a.stages;
    constexpr int kSfSlots = grp_slots<F>();
    static_assert(kSfSlots % sf_groups<F>() == 0 && kSfSlots <= 8, "a slot belongs to one group");
    unsigned char* sA = base;
    unsigned char* sB = sA + ns * kPairABytes;
    unsigned char* sS = sB + ns * kPairBBytes;  // scale chunks: the weights', then the tokens'
    unsigned char* sR = sS + kSfSlots * kGrpSfBytes;  // chunks of the residual
    Group* groups = reinterpret_cast<Group*>(sR + a.res_area);
    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int rank = (int)uniform(cluster_rank());
    const int first = (int)(blockIdx.x >> 1), step = (int)(gridDim.x >> 1);
    if (threadIdx.x == 0) {
        for (int w = 0; w < 8; ++w)
            for (int b = 0; b < kResSlots; ++b) bar_init(&s_res[w][b], 1);
        for (int s = 0; s < ns; ++s) {
            bar_init(&sh.full[s], chunk_is_stage<F>() ? 9 : 1);
            bar_init(&sh.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(&sh.acc_full[b], 1);
            bar_init(&sh.acc_empty[b], 16);
        }
        for (int b = 0; b < kSfSlots; ++b) {
            bar_init(&sh.sf_full[b], a.ts_wide ? 1 : 33);  // TMA's, and each lane's of warp 10
            bar_init(&sh.sf_empty[b], 4);
        }
        for (int b = 0; b < kSfBufs; ++b) {
            bar_init(&sh.sf_ready[b], 8);
            bar_init(&sh.sf_free[b], 1);
        }
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
        group_table<kTokTile>(groups, a.offs, a.G, a.rows, lane);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are set up
    tc_fence_after();
    const uint32_t tmem = uniform(sh.tmem);
    const int tiles = groups[a.G].tile * a.tiles_n;
    GroupedTile w;
    w.g = 0;
    bool bad = false;
    if (warp == 0) {
        const bool elected = elect_lane();
        const uint32_t full0 = map_rank(smem_u32(&sh.full[0]), 0);
        Ring r;
        uint32_t g = 0;
        for (int t = first; t < tiles && !bad; t += step) {
            grouped_tile(a, groups, t, w);
            const int half = w.cols >> 1;  // tokens of this CTA
            const int32_t bt = w.t0 + half * rank, an = w.g * a.N + w.n0 + 128 * rank;
            const uint32_t bytes = (uint32_t)(2 * (kPairABytes + half * kRowBytes));
            for (int i = 0; i < a.nkb; ++i) {
                const int s = r.slot;
                if (g >= (uint32_t)ns && !warp_wait<Sync::CLUSTER>(&sh.empty[s], r.parity ^ 1u)) {
                    bad = true;
                    break;
                }
                const uint32_t bar = full0 + 8 * s;
                unsigned char *pa = sA + s * kPairABytes, *pb = sB + s * kPairBBytes;
                if (elected) {
                    if (rank == 0) mbar_expect_tx(&sh.full[s], bytes);
                    pair_load_2d(pa, &a.tw, i * kRowBytes, an, bar);
                    if (half == kTokTile / 2) {
                        pair_load_2d(pb, &a.tt, i * kRowBytes, bt, bar);
                    } else {
                        for (int j = 0; j < half; j += kTokBox)
                            pair_load_2d(pb + j * kRowBytes, &a.tt16, i * kRowBytes, bt + j, bar);
                    }
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
            int j = 0;
            for (int t = first; t < tiles && !bad; t += step, ++j) {
                grouped_tile(a, groups, t, w);
                const uint32_t id = idesc<F>(kPairM, (int)uniform(w.cols), 0);
                const int ab = j & 1;
                if (j >= 2 && !warp_wait<Sync::TENSOR>(&sh.acc_empty[ab], (uint32_t)((j >> 1) - 1) & 1)) {
                    bad = true;
                    break;
                }
                const uint32_t acc = tmem + (uint32_t)(ab * kTokTile);
                for (int i = 0; i < a.nkb; ++i) {
                    const int s = r.slot, in_chunk = i % chunk_stages<F>();
                    if ((!chunk_is_stage<F>() && in_chunk == 0 &&
                         !warp_wait<Sync::TENSOR>(&sh.sf_ready[f.slot], f.parity)) ||
                        (!warp_agrees(here) && !warp_wait<Sync::CLUSTER>(&sh.full[s], r.parity))) {
                        bad = true;
                        break;
                    }
                    r.next(ns);
                    tc_fence_after();
                    const int nk = min(F::kSfTiles, a.kb - F::kSfTiles * i);
                    const uint32_t a0 = desc_lo(smem_u32(sA) + s * kPairABytes);
                    const uint32_t b0 = desc_lo(smem_u32(sB) + s * kPairBBytes);
                    const uint32_t sf = tmem + kPairSfCol + f.slot * kSfCols;
                    const bool last = in_chunk == chunk_stages<F>() - 1 || i + 1 == a.nkb;
                    if (elected) {
                        grouped_stage<F>(acc, a0, b0, id, sf + 4 * in_chunk, sf + 16 + 6 * in_chunk, nk, i > 0);
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
            grouped_tile(a, groups, t, w);
            const int32_t ra = w.g * a.row_tiles + (w.n0 >> 7) + rank;
            const uint8_t* src = a.ts + w.t0 * a.ts_pitch;
            for (int k = 0; k < a.kb; k += kSfChunkTiles) {
                if (chunks >= (uint32_t)kSfSlots && !warp_wait(&sh.sf_empty[f.slot], f.parity ^ 1u)) {
                    bad = true;
                    break;
                }
                unsigned char* ps = sS + f.slot * kGrpSfBytes;
                uint64_t* bar = &sh.sf_full[f.slot];
                unsigned char* pt = ps + kSfChunkA;
                if (elected) {
                    const int boxes = w.cols > kTokTile / 2 ? 6 : w.cols >> 5;
                    mbar_expect_tx(bar, (uint32_t)(kSfChunkA + (a.ts_wide ? 512 * boxes : 0)));
                    sf_load_3d(ps, &a.tsw, k, ra, bar);
                    if (a.ts_wide) {
                        if (boxes == 6) tma_load_2d(pt, &a.tst, 4 * k, w.t0, bar);
                        else
                            for (int j = 0; j < boxes; ++j)
                                tma_load_2d(pt + 512 * j, &a.tst32, 4 * k, w.t0 + 32 * j, bar);
                    }
                }
                __syncwarp();
                if (!a.ts_wide) {
                    for (int r = lane; r < w.live; r += 32) {
                        const uint8_t* p = src + r * a.ts_pitch + 4 * k;
                        for (int j = 0; j < min(kSfChunkTiles, a.kb - k); ++j)
                            cp_async4(smem_u32(pt) + 16 * r + 4 * j, p + 4 * j);
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
    } else if (warp < 6 || (sf_groups<F>() == 2 && warp > 10 && warp < 15)) {
        // scales: lane l of quadrant q writes the weights' (rows l, 32 + l, .. in the words
        // of tile kk) to columns 4 kk ..., the tokens' (token 32 i + l, tiles in the words)
        // to columns 16 + 6 kk ...
        const int q = warp & 3;
        const uint32_t lane_base = tmem + kPairSfCol + ((uint32_t)(32 * q) << 16);
        const uint32_t full0 = map_rank(smem_u32(&sh.full[0]), 0);
        const uint32_t ready0 = map_rank(smem_u32(&sh.sf_ready[0]), 0);
        Ring f, d;          // shared-memory slots; tensor-memory buffers
        Ring r, u;          // chunk_is_stage: its stage; the one whose buffer it takes over
        const uint32_t mine = warp < 6 ? 0u : 1u;  // the group of scale warps
        uint32_t chunks = 0;
        for (int t = first; t < tiles && !bad; t += step) {
            for (int i = 0; i < a.nkb; i += chunk_stages<F>()) {
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
                const unsigned char* ps = sS + f.slot * kGrpSfBytes + 16 * lane;
                uint32_t va[16], vb[24];
#pragma unroll
                for (int kk = 0; kk < kSfChunkTiles; ++kk) {
                    const uint4 x = *reinterpret_cast<const uint4*>(ps + kk * kSfTileBytes);
                    va[4 * kk] = x.x; va[4 * kk + 1] = x.y; va[4 * kk + 2] = x.z; va[4 * kk + 3] = x.w;
                }
#pragma unroll
                for (int j = 0; j < 6; ++j) {
                    const uint4 x = *reinterpret_cast<const uint4*>(ps + kSfChunkA + j * 512);
                    vb[j] = x.x; vb[6 + j] = x.y; vb[12 + j] = x.z; vb[18 + j] = x.w;
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
                    // behind the stores that use its values (k_linear_pair)
                    bar_arrive(&sh.sf_empty[f.slot]);
                }
                r.next(ns);
                ++chunks;
                f.next(kSfSlots);
                d.next(kSfBufs);
            }
        }
    } else {
        // quadrant, and which of the two warps of it
        const int q = warp & 3, half = warp < 10 ? 0 : 1, e = 4 * half + q;
        const bool pre = a.ep.pre != nullptr;
        int j = 0;
        // The residual's chunks come kResSlots - 1 ahead of the sums, over the ends of tiles: a
        // walk of their own (1590 tokens of 11 experts x 13696 x 1024 NVFP4 57 us, with loads into
        // registers one chunk ahead 64; 5717 x 7728 x 960 fp32 84, 97).
        uint32_t rc = 0, fc = 0;  // chunks added, fetched
        int ft = first, f0 = kEpiTok * half;
        GroupedTile f = w;
        unsigned char* bufs = sR + e * kResSlots * kResBytes;
        auto fetch = [&] {
            for (; ft < tiles; ft += step) {
                if (f0 == kEpiTok * half) grouped_tile(a, groups, ft, f);
                const int n = f.n0 + 128 * rank + 32 * q;
                if (n >= a.N) continue;
                if (lane == 0) {
                    const uint32_t s = fc % kResSlots;
                    mbar_expect_tx(&s_res[e][s], kResBytes);
                    tma_load_2d(bufs + s * kResBytes, &a.tres, n, f.t0 + f0, &s_res[e][s]);
                }
                ++fc;
                f0 += 2 * kEpiTok;
                if (f0 >= f.cols) {
                    f0 = kEpiTok * half;
                    ft += step;
                }
                return;
            }
        };
        if (a.ep.residual)
            for (int i = 0; i + 1 < kResSlots; ++i) fetch();
        // What a tile's sums take besides, asked for while the tile before it is finished
        // (1590 x 13696 x 1024 as above 55 us instead of 57, without a residual 37.9, 39.2).
        GroupedTile next = w;
        float next_bias = 0.0f, b_amax = 0.0f, a_amax = 0.0f;
        auto ask = [&](int t) {
            grouped_tile(a, groups, t, next);
            const int n = next.n0 + 128 * rank + 32 * q + lane;
            if (a.ep.bias && n < a.N) {
                const int64_t i = (int64_t)next.g * a.N + n;
                next_bias = a.ep.bias32 ? ld_f32(static_cast<const float*>(a.ep.bias) + i)
                                        : raw_value<OT>(ld_raw<OT>(a.ep.bias, i));
            }
            if constexpr (F::kGlobal) {
                b_amax = ld_f32(a.ep.b_amax + next.g);
                if (!a.ep.a_row) a_amax = ld_f32(a.ep.a_amax + next.g);
            }
        };
        if (first < tiles) ask(first);
        for (int t = first; t < tiles; t += step, ++j) {
            w = next;
            const bool res = a.ep.residual && w.n0 + 128 * rank + 32 * q < a.N;
            const int n = w.n0 + 128 * rank + 32 * q + lane;
            const bool in = n < a.N;
            // column n of the tile's rows; rows of this lane (none past the weights)
            const int64_t at = (int64_t)w.t0 * a.N + n;
            const int live = in ? w.live : 0;
            const float bias = next_bias;
            float gb = 1.0f, ga0 = 1.0f;
            if constexpr (F::kGlobal) {
                gb = fdiv(1.0f, global_scale(b_amax, a.ep.six_bound));
                if (a.ep.a_row) {
                    for (int c = lane; c < w.live; c += 32)
                        s_ga[e][c] = fdiv(1.0f, global_scale(ld_f32(a.ep.a_amax + w.t0 + c), a.ep.six_bound));
                } else {
                    ga0 = fdiv(1.0f, global_scale(a_amax, a.ep.six_bound));
                }
            }
            if (t + step < tiles) ask(t + step);
            const int ab = j & 1;
            if (!bad && !warp_wait<Sync::TENSOR>(&sh.acc_full[ab], (uint32_t)(j >> 1) & 1)) bad = true;
            __syncwarp();
            tc_fence_after();
            for (int c0 = kEpiTok * half; c0 < w.cols; c0 += 2 * kEpiTok) {
                uint32_t u[kEpiTok];
                tmem_ld16(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(ab * kTokTile + c0), u);
                if (c0 + 2 * kEpiTok >= w.cols) {  // this warp has read the accumulator
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) cluster_arrive(map_rank(smem_u32(&sh.acc_empty[ab]), 0));
                }
                float v[kEpiTok];
#pragma unroll
                for (int i = 0; i < kEpiTok; ++i) v[i] = __uint_as_float(u[i]);
                if constexpr (F::kGlobal) {
                    if (a.ep.a_row) {
#pragma unroll
                        for (int i = 0; i < kEpiTok / 4; ++i) {
                            const float4 ga = *reinterpret_cast<const float4*>(&s_ga[e][c0 + 4 * i]);
                            v[4 * i] = fmul(fmul(v[4 * i], ga.x), gb);
                            v[4 * i + 1] = fmul(fmul(v[4 * i + 1], ga.y), gb);
                            v[4 * i + 2] = fmul(fmul(v[4 * i + 2], ga.z), gb);
                            v[4 * i + 3] = fmul(fmul(v[4 * i + 3], ga.w), gb);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < kEpiTok; ++i) v[i] = fmul(fmul(v[i], ga0), gb);
                    }
                }
                if (a.ep.bias) {
#pragma unroll
                    for (int i = 0; i < kEpiTok; ++i) v[i] = fadd(v[i], bias);
                }
                constexpr int kElt = OT == Out::F32 ? 4 : 2;
                const int64_t to = (at + (int64_t)c0 * a.N) * kElt;
                if (pre) store_column<OT>(static_cast<char*>(a.ep.pre) + to, a.N, v, live - c0);
                act_apply<OT>(a.ep.act, v);
                if (res) {
                    const uint32_t s = rc % kResSlots;
                    // (also once a wait gave up: no copy is in flight when the CTA leaves)
                    if (!warp_wait(&s_res[e][s], (rc / kResSlots) & 1u)) bad = true;
                    const unsigned char* buf = bufs + s * kResBytes;
#pragma unroll
                    for (int i = 0; i < kEpiTok; ++i)
                        v[i] = fadd(v[i], raw_value<OT>(OT == Out::F32 ? reinterpret_cast<const uint32_t*>(buf)[32 * i + lane]
                                                                       : reinterpret_cast<const unsigned short*>(buf)[32 * i + lane]));
                    ++rc;
                    // read before the slot is filled again
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    fetch();
                }
                store_column<OT>(static_cast<char*>(a.ep.out) + to, a.N, v, live - c0);
            }
            __syncwarp();  // the decode scales are read before the next tile's replace them
        }
    }
    // every MMA issued has completed before the tensor memory is freed
    if (warp == 1 && !warp_wait<Sync::TENSOR>(&sh.done, 0)) bad = true;
    if (bad) sh.fail = 1;
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other may touch its memory
    if (sh.fail && threadIdx.x == 0 && first < tiles) {
        grouped_tile(a, groups, first, w);
        store_out<OT>(a.ep.out, (int64_t)w.t0 * a.N + w.n0, __int_as_float(0x7FC00000));
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kAllColumns) : "memory");
    }
}

// ------------------------------------------------------------------ out[e] = a[:, e] . b[:, e]^T
// k_grouped_wgrad: a and b are column-wise 8-bit forms whose columns are the tokens,
// each group's part a whole number of 128 (a stage, a scale tile); tiles of 256 x 192 of
// out[e] with as many stages as the group has columns / 128, none for an empty
// group, whose product is 0.  The rest is k_linear_pair's, but for the last rows of
// out[e], behind which the next group's lie: a chunk of 32 rows that ends there is
// copied row by row.
// With a thousand tokens an expert a tile has eight or nine stages, and 96 KB of fp32 an
// SM leave for every 250 KB that come.  8 x 14336 x 4096 of 8192 tokens 438 us, 323 of
// them without the stores and 307 without the chunks either; operands and stores
// together are 15 TB/s through L2.  Measured and not kept: more chunk buffers and fewer
// stages, 490 .. 516 us; rows stored from registers by whole sectors with seven stages, 520;
// L2 priorities for the stores and the operands, 438.
// With a residual a warp has four chunks and fetches three ahead, over the ends of tiles
// (one chunk ahead in two: 8 x 14336 x 4096 950 us, 64 x 2048 x 1408 of 4096 tokens 342;
// two ahead in three 724, 263; three ahead in four 650, 232, 6.4 TB/s).
struct WgradArgs {
    CUtensorMap ta;    // a codes, box 128 bytes x 128 rows
    CUtensorMap tb;    // b codes, box 128 bytes x 96 rows
    CUtensorMap tsa;   // tiled scales, box 1 x 4 x 512
    CUtensorMap tsb;   // box 2 x 4 x 512
    CUtensorMap tout;  // out, residual [G * M, N]: box 128 bytes x 32 rows
    CUtensorMap tres;
    Epilogue ep;       // residual, out
    const int32_t* offs;
    int G;
    int rows;              // packed rows
    int M, N;              // of out[e]
    int tiles_m, tiles_n;
    int band;
    int stages;
};

struct WgradTile {
    int g;
    int32_t m0, m_end;   // rows of a, and of out from out_row; where they end
    int32_t n0;
    int32_t k0, nkb;     // first stage of the columns, stages
    int32_t out_row;
};

__device__ __forceinline__ void wgrad_tile(const WgradArgs& a, const Group* t, int tile, WgradTile& w) {
    const int per_group = a.tiles_m * a.tiles_n;
    const int g = tile / per_group, r0 = tile - g * per_group;
    const int per_band = a.band * a.tiles_n;
    const int band = r0 / per_band, r = r0 - band * per_band;
    const int rows = min(a.band, a.tiles_m - band * a.band);
    const int col = r / rows;
    w.g = g;
    w.m0 = (band * a.band + r - col * rows) * kPairM;
    w.m_end = a.M;
    w.n0 = col * kPairN;
    w.k0 = t[g].tile;
    w.nkb = t[g + 1].tile - w.k0;
    w.out_row = g * a.M;
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

// Chunks of a warp of the epilogue in shared memory.
template <bool kRes> constexpr int wgrad_slots() { return kRes ? 4 : 2; }

template <Out OT, bool kRes>
__global__ void __launch_bounds__(pair_threads<F8>(), 1) k_grouped_wgrad(const __grid_constant__ WgradArgs a) {
    using F = F8;
    extern __shared__ __align__(1024) unsigned char s_raw[];
    __shared__ PairShared sh;
    constexpr int kSlots = wgrad_slots<kRes>();
    __shared__ __align__(8) uint64_t s_res[4][kSlots];  // the residual's chunks are here
    unsigned char* base = s_raw + ((1024u - (smem_u32(s_raw) & 1023u)) & 1023u);
    const int ns = a.stages;
    constexpr int kSfSlots = sf_slots<F>();
    unsigned char* sA = base;
    unsigned char* sB = sA + ns * kPairABytes;
    unsigned char* sC = sB + ns * kPairBBytes;          // epilogue chunks
    unsigned char* sS = sC + 4 * kSlots * kChunkBytes;  // scale chunks: a, then b's two row tiles
    Group* groups = reinterpret_cast<Group*>(sS + kSfSlots * kSfChunkBytes);
    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int rank = (int)uniform(cluster_rank());
    const int first = (int)(blockIdx.x >> 1), step = (int)(gridDim.x >> 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < ns; ++s) {
            bar_init(&sh.full[s], 1);
            bar_init(&sh.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(&sh.acc_full[b], 1);
            bar_init(&sh.acc_empty[b], 8);
        }
        for (int b = 0; b < kSfSlots; ++b) {
            bar_init(&sh.sf_full[b], 1);
            bar_init(&sh.sf_empty[b], 4);
        }
        for (int b = 0; b < kSfBufs; ++b) {
            bar_init(&sh.sf_ready[b], 8);
            bar_init(&sh.sf_free[b], 1);
        }
        for (int w = 0; w < 4; ++w)
            for (int b = 0; b < kSlots; ++b) bar_init(&s_res[w][b], 1);
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
        group_table<kRowBytes>(groups, a.offs, a.G, a.rows, lane);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are set up
    tc_fence_after();
    const uint32_t tmem = uniform(sh.tmem);
    const int tiles = a.G * a.tiles_m * a.tiles_n;
    WgradTile w;
    w.g = 0;
    bool bad = false;
    if (warp == 0) {
        const bool elected = elect_lane();
        const uint32_t full0 = map_rank(smem_u32(&sh.full[0]), 0);
        Ring r;
        uint32_t g = 0;
        for (int t = first; t < tiles && !bad; t += step) {
            wgrad_tile(a, groups, t, w);
            const int32_t am = w.m0 + 128 * rank;
            const int32_t bn = w.n0 + 96 * rank;
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
                    if (rank == 0) mbar_expect_tx(&sh.full[s], (uint32_t)(2 * kPairStageBytes));
                    pair_load_2d(pa, &a.ta, x, am, bar);
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
                wgrad_tile(a, groups, t, w);
                if (w.nkb == 0) continue;  // no accumulator: the epilogue takes zeros
                const int ab = j & 1;
                if (j >= 2 && !warp_wait<Sync::TENSOR>(&sh.acc_empty[ab], (uint32_t)((j >> 1) - 1) & 1)) {
                    bad = true;
                    break;
                }
                ++j;
                const uint32_t acc = tmem + (uint32_t)(ab * kPairN);
                for (int i = 0; i < w.nkb; ++i) {
                    const int s = r.slot, in_chunk = i % chunk_stages<F>();
                    if ((in_chunk == 0 && !warp_wait<Sync::TENSOR>(&sh.sf_ready[f.slot], f.parity)) ||
                        (!warp_agrees(here) && !warp_wait<Sync::CLUSTER>(&sh.full[s], r.parity))) {
                        bad = true;
                        break;
                    }
                    r.next(ns);
                    tc_fence_after();
                    const uint32_t a0 = desc_lo(smem_u32(sA) + s * kPairABytes);
                    const uint32_t b0 = desc_lo(smem_u32(sB) + s * kPairBBytes);
                    const uint32_t sf = tmem + kPairSfCol + f.slot * kSfCols;
                    const bool last = in_chunk == chunk_stages<F>() - 1 || i + 1 == w.nkb;
                    if (elected) {
                        pair_stage<F>(acc, a0, b0, sf + 4 * in_chunk, sf + 16 + 6 * in_chunk, 1, i > 0);
                        pair_commit(&sh.empty[s]);
                        if (last) pair_commit(&sh.sf_free[f.slot]);
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
            wgrad_tile(a, groups, t, w);
            const int32_t ra = (w.m0 + 128 * rank) >> 7, rb = w.n0 >> 7;
            for (int k = 0; k < w.nkb; k += kSfChunkTiles) {
                if (chunks >= (uint32_t)kSfSlots && !warp_wait(&sh.sf_empty[f.slot], f.parity ^ 1u)) {
                    bad = true;
                    break;
                }
                unsigned char* ps = sS + f.slot * kSfChunkBytes;
                uint64_t* bar = &sh.sf_full[f.slot];
                if (elected) {
                    mbar_expect_tx(bar, (uint32_t)kSfChunkBytes);
                    sf_load_3d(ps, &a.tsa, w.k0 + k, ra, bar);
                    sf_load_3d(ps + kSfChunkA, &a.tsb, w.k0 + k, rb, bar);
                }
                __syncwarp();
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
    } else if (warp < 6) {
        // scales: lane l of quadrant q writes row l of each 16-byte-wide tile, as in
        // k_linear_pair
        const int q = warp & 3;
        const uint32_t lane_base = tmem + kPairSfCol + ((uint32_t)(32 * q) << 16);
        const uint32_t ready0 = map_rank(smem_u32(&sh.sf_ready[0]), 0);
        Ring f, d;          // shared-memory slots; tensor-memory buffers
        uint32_t chunks = 0;
        for (int t = first; t < tiles && !bad; t += step) {
            wgrad_tile(a, groups, t, w);
            const bool half = (w.n0 & 127) != 0;  // b starts half-way into a scale tile
            for (int i = 0; i < w.nkb; i += chunk_stages<F>()) {
                if (!warp_wait(&sh.sf_full[f.slot], f.parity)) {
                    bad = true;
                    break;
                }
                const unsigned char* ps = sS + f.slot * kSfChunkBytes + 16 * lane;
                uint32_t va[16], vb[24];
#pragma unroll
                for (int kk = 0; kk < kSfChunkTiles; ++kk) {
                    const uint4 x = *reinterpret_cast<const uint4*>(ps + kk * kSfTileBytes);
                    const uint4 y = *reinterpret_cast<const uint4*>(ps + kSfChunkA + kk * kSfTileBytes);
                    const uint4 z = *reinterpret_cast<const uint4*>(ps + 2 * kSfChunkA + kk * kSfTileBytes);
                    va[4 * kk] = x.x; va[4 * kk + 1] = x.y; va[4 * kk + 2] = x.z; va[4 * kk + 3] = x.w;
                    vb[6 * kk] = half ? y.z : y.x;
                    vb[6 * kk + 1] = half ? y.w : y.y;
                    vb[6 * kk + 2] = half ? z.x : y.z;
                    vb[6 * kk + 3] = half ? z.y : y.w;
                    vb[6 * kk + 4] = half ? z.z : z.x;
                    vb[6 * kk + 5] = half ? z.w : z.y;
                }
                if (chunks >= (uint32_t)kSfBufs) {
                    // the MMAs that read this buffer are done
                    if (!warp_wait<Sync::TENSOR>(&sh.sf_free[d.slot], d.parity ^ 1u)) {
                        bad = true;
                        break;
                    }
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
                    cluster_arrive(ready0 + 8 * d.slot);
                    // behind the stores that use its values (k_linear_pair)
                    bar_arrive(&sh.sf_empty[f.slot]);
                }
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
        unsigned char* bufs = sC + e * kSlots * kChunkBytes;  // for out and the residual
        uint32_t c = 0;  // chunks of this warp
        int j = 0;       // accumulators used
        // The residual's chunks come kSlots - 1 ahead of the sums, over the ends of tiles: a walk
        // of their own.
        uint32_t fc = 0;
        int ft = first, fk = 0;
        WgradTile f = w;
        auto fetch = [&] {
            for (; ft < tiles; ft += step) {
                if (fk == 0) wgrad_tile(a, groups, ft, f);
                const int32_t row = f.m0 + 128 * rank + 32 * q;
                if (row >= f.m_end) continue;
                if (lane == 0) {
                    const uint32_t s = fc % kSlots;
                    mbar_expect_tx(&s_res[e][s], kChunkBytes);
                    tma_load_2d(bufs + s * kChunkBytes, &a.tres, f.n0 + fk * kCols, f.out_row + row, &s_res[e][s]);
                }
                ++fc;
                if (++fk == kChunks) {
                    fk = 0;
                    ft += step;
                }
                return;
            }
        };
        if constexpr (kRes) {
            for (int i = 0; i + 1 < kSlots; ++i) fetch();
        }
        for (int t = first; t < tiles; t += step) {
            wgrad_tile(a, groups, t, w);
            const int32_t mw = w.m0 + 128 * rank + 32 * q;           // first row of this warp
            const int live = max(0, min(32, w.m_end - mw));          // rows of the group
            const int32_t orow = w.out_row + mw;
            if (kRes && OT == Out::F32 && t + step < tiles && lane < kChunks) {
                // The next tile's residual on its way to L2: three chunks are half a tile of
                // 32 bits (two ahead 264 us instead of 295), but a whole one of 16 (76.5, 74.7
                // without, 16 x 2048 x 2048).
                WgradTile x = w;
                wgrad_tile(a, groups, t + step, x);
                const int32_t row = x.m0 + 128 * rank + 32 * q;
                if (row < x.m_end && x.n0 + lane * kCols < a.N)
                    prefetch_chunk(&a.tres, x.n0 + lane * kCols, x.out_row + row);
            }
            const bool sum = w.nkb > 0;  // there is a product
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
                const uint32_t s = c % kSlots;
                const uint32_t buf = smem_u32(bufs + s * kChunkBytes);
                // (also once a wait gave up: no copy is in flight when the CTA leaves)
                if (kRes && !warp_wait(&s_res[e][s], (c / kSlots) & 1u)) bad = true;
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
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
                    constexpr int kPieces = 32 * kElt / 16;
                    if (kRes) add_pieces<OT>(buf + lane * 128, lane, kPieces * h, v);
                    put_pieces<OT>(buf + lane * 128, lane, kPieces * h, v);
                }
                const int32_t n = w.n0 + k * kCols;
                if (live < 32) {  // the rows below are another group's
                    __syncwarp();
                    copy_rows<OT>(buf, a.ep.out, orow, n, a.N, live, lane);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0 && live == 32) store_chunk(&a.tout, n, orow, buf);
                if (lane == 0) {
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    // the chunk before this one has left its slot, which the next one takes
                    // (or the next one to be fetched)
                    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kRes ? 1 : kSlots - 1) : "memory");
                }
                if constexpr (kRes) fetch();
            }
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
        wgrad_tile(a, groups, first, w);
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
