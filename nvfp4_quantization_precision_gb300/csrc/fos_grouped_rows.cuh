// fos_grouped_rows.cuh -- the grouped product for few tiles: k_grouped (fos_grouped.cuh)
// keeps two SMs on all of K for a tile of 256 weight rows, and with few tokens or
// narrow weights most SMs have none.  Here a CTA takes 128 weight rows x nt <= 64 tokens
// of one group, and the S CTAs of a cluster split K and add their partial tiles in
// rank order: k_linear_rows, whose roles, ring, waits and epilogue these are, with
//   tiles    from the table of groups (fos_groups.cuh): t = (chunk of 64 tokens of a
//            group, 128 weight rows), walked by t, t + clusters, ...
//   scales   of the tokens plain: warp 6 copies a stage's words, four bytes a token and
//            scale tile, to their places in a tile of 512 bytes by cp.async, three stages
//            ahead of the arrival that hands them to the copies into tensor memory
// A tile may start at any row: rows of the next group in its box are columns that
// nobody reads.
// Bound by latency: with one tile a CTA the launch, the first stage's way in, stages / S
// times 0.32 us (NVFP4 0.37) and the sums.  Measured (GPU us; k_grouped): 8 bit, 2 tokens of
// 2 of 17 experts x 320 x 8192 7.4 (18.3), 4 tokens of 4 of 10 x 1104 x 10496 13.0 (23.0), a token
// x 4096 x 14336 14.8 (29.1); NVFP4, a token x 1104 x 8512 6.4 (18.5), 7 tokens of 7 x 896 x 12480
// 13.8 (25.5).
#pragma once

#include "fos_grouped.cuh"

namespace fos {
namespace lin {

constexpr int kGrpRowsTok = 64;  // tokens of a chunk
constexpr int kGrpRowsLag = 3;   // stages of the tokens' scales on their way
static_assert(kGrpRowsLag < kSfRing, "the ring of stages is longer");

struct GroupedRowsArgs {
    CUtensorMap tp;      // weights' codes, box 128 bytes x 128 rows, the groups' below one another
    CUtensorMap tq;      // tokens' codes, box 128 bytes x nt rows
    const uint8_t* sfp;  // weights' tiled scales
    const uint8_t* sfq;  // plain scales of the tokens
    int64_t sfq_pitch;   // bytes of a row of them
    Epilogue ep;
    const int32_t* offs;
    int G;
    int rows;            // packed rows
    int N;               // weight rows of a group
    int tiles_p;         // tiles of 128 of them
    int kb, nkb;         // scale tiles and stages along K
    int nt;
    int splits;
    int stages;
};

template <class F, Out OT>
__global__ void __launch_bounds__(kRowsThreads, 1) k_grouped_rows(const __grid_constant__ GroupedRowsArgs a) {
    extern __shared__ __align__(1024) unsigned char s_raw[];
    __shared__ RowsShared sh;
    __shared__ float s_ga[F::kGlobal ? kGrpRowsTok : 1];  // the tokens' decode scales
    unsigned char* base = s_raw + ((1024u - (smem_u32(s_raw) & 1023u)) & 1023u);
    const int nt = a.nt, S = a.splits, ns = a.stages;
    const int qbytes = nt * kRowBytes;
    constexpr int kPBytes = 128 * kRowBytes, kSf = F::kSfTiles * kSfTileBytes;
    unsigned char* sP = base;
    unsigned char* sQ = sP + ns * kPBytes;
    unsigned char* sFP = sQ + ns * qbytes;
    unsigned char* sFQ = sFP + ns * kSf;
    Group* groups = reinterpret_cast<Group*>(sFQ + ns * kSf);
    float* red = reinterpret_cast<float*>(base);  // [nt][128] partial tile, over the ring
    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int rank = S > 1 ? (int)uniform(cluster_rank()) : 0;
    const int first = (int)blockIdx.x / S, step = (int)gridDim.x / S;
    // this CTA's stages of every tile
    const int k_lo = a.nkb * rank / S, k_hi = a.nkb * (rank + 1) / S;
    if (warp == 0) {
        if (lane < ns) {
            bar_init(&sh.full[lane], 3);  // codes, the weights' scales, the tokens'
            bar_init(&sh.empty[lane], 1);
        } else if (lane == 31) {
            bar_init(&sh.acc_full, 1);
            bar_init(&sh.done, 1);
            sh.fail = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const bool elected = elect_lane();
    uint32_t g = 0;   // stages loaded (warps 0, 6) or consumed (warp 1) so far
    Ring r, w;        // the stage in work; warp 1: the one whose scales are overwritten
    bool bad = false;
    bool here = false, free = false;  // warp 1: the next stage is full, its scale buffer is free
    int j = 0;        // tiles of this CTA so far
    __syncwarp();
    chain_wait();
    chain_release();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh.tmem)), "r"(kAllColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (warp == 6) {
        group_table<kGrpRowsTok>(groups, a.offs, a.G, a.rows, lane);
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(sh.tmem);
    const int tiles = groups[a.G].tile * a.tiles_p;
    int e = 0;  // the tile's group
    for (int t = first; t < tiles; t += step, ++j) {
        const int chunk = t / a.tiles_p, n0 = (t - chunk * a.tiles_p) * 128;
        e = group_of(groups, a.G, chunk, e);
        const int m0 = groups[e].row + (chunk - groups[e].tile) * kGrpRowsTok;
        const int mt = min(nt, groups[e + 1].row - m0);  // tokens of the tile
        if (warp == 0) {
            for (int i = k_lo; i < k_hi && !bad; ++i) {
                const int s = r.slot;
                if (g >= (uint32_t)ns && !warp_wait(&sh.empty[s], r.parity ^ 1u)) {
                    bad = true;
                    break;
                }
                if (elected) {
                    mbar_expect_tx(&sh.full[s], (uint32_t)(kPBytes + qbytes));
                    tma_load_2d(sP + s * kPBytes, &a.tp, i * kRowBytes, e * a.N + n0, &sh.full[s]);
                    tma_load_2d(sQ + s * qbytes, &a.tq, i * kRowBytes, m0, &sh.full[s]);
                }
                __syncwarp();
                ++g;
                r.next(ns);
            }
        } else if (warp == 6) {
            const uint8_t* pp = a.sfp + (((int64_t)e * ((a.N + 127) >> 7) + (n0 >> 7)) * a.kb + F::kSfTiles * k_lo) *
                                            kSfTileBytes;
            Ring in = r;  // the stage whose words are next to have arrived
            auto hand_over = [&] {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) bar_arrive(&sh.full[in.slot]);
                in.next(ns);
            };
            int late = 0;  // stages not handed over
            for (int i = k_lo; i < k_hi; ++i) {
                const int s = r.slot;
                if (g >= (uint32_t)ns && !warp_wait(&sh.empty[s], r.parity ^ 1u)) {
                    bad = true;
                    break;
                }
                const int nk = min(F::kSfTiles, a.kb - F::kSfTiles * i);
                if (elected) {
                    mbar_expect_tx(&sh.full[s], (uint32_t)(nk * kSfTileBytes));
                    bulk_load(sFP + s * kSf, pp, (uint32_t)(nk * kSfTileBytes), &sh.full[s]);
                }
                __syncwarp();
                pp += kSf;
                const uint32_t dq = smem_u32(sFQ) + s * kSf;
                for (int c = lane; c < mt; c += 32) {
                    const uint8_t* p = a.sfq + (m0 + c) * a.sfq_pitch + 4 * F::kSfTiles * i;
#pragma unroll
                    for (int kk = 0; kk < F::kSfTiles; ++kk)
                        if (kk < nk) cp_async4(dq + kk * kSfTileBytes + 16 * (c & 31) + 4 * (c >> 5), p + 4 * kk);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                ++g;
                r.next(ns);
                if (++late > kGrpRowsLag) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(kGrpRowsLag) : "memory");
                    hand_over();
                    --late;
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            for (; late > 0; --late) hand_over();
        } else if (warp == 1) {
            for (int i = k_lo; i < k_hi && !bad; ++i) {
                const int s = r.slot;
                const bool over = g >= (uint32_t)kSfRing;  // a scale buffer is used again
                if ((!warp_agrees(here) && !warp_wait(&sh.full[s], r.parity)) ||
                    (over && !warp_agrees(free) && !warp_wait(&sh.empty[w.slot], w.parity))) {
                    bad = true;
                    break;
                }
                if (over) w.next(ns);
                r.next(ns);
                here = mbar_ask(&sh.full[r.slot], r.parity);
                free = mbar_ask(&sh.empty[w.slot], w.parity);
                tc_fence_after();
                const int nk = min(F::kSfTiles, a.kb - F::kSfTiles * i);
                const uint32_t sfp = tmem + 256 + (g % kSfRing) * 48, sfq = sfp + 4 * F::kSfTiles;
                if (elected) {
                    rows_stage<F, 1>(tmem, desc_lo(smem_u32(sP) + s * kPBytes), desc_lo(smem_u32(sQ) + s * qbytes),
                                     idesc<F>(128, nt, 0), sfp, sfq, sf_desc_lo(smem_u32(sFP) + s * kSf),
                                     sf_desc_lo(smem_u32(sFQ) + s * kSf), nk, i > k_lo);
                    tc_commit(&sh.empty[s]);
                }
                __syncwarp();
                ++g;
            }
            if (!bad && elected) tc_commit(&sh.acc_full);
            __syncwarp();
        } else {
            const int q = warp & 3, ew = warp - 2;
            // finishing, lane l has weight rows 4 l .. 4 l + 3 of the tile
            const int64_t n = n0 + 4 * lane;
            const bool nin = n < a.N;
            float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (a.ep.bias && nin) {
                const int64_t at = (int64_t)e * a.N + n;
                if (a.ep.bias32) load4<Out::F32>(a.ep.bias, at, bias);
                else load4<OT>(a.ep.bias, at, bias);
            }
            float gb = 1.0f;
            if constexpr (F::kGlobal) {
                gb = fdiv(1.0f, global_scale(ld_f32(a.ep.b_amax + e), a.ep.six_bound));
                for (int c = 32 * ew + lane; c < mt; c += 128)
                    s_ga[c] = fdiv(1.0f, global_scale(ld_f32(a.ep.a_amax + (a.ep.a_row ? m0 + c : e)), a.ep.six_bound));
            }
            if (!bad && !warp_wait(&sh.acc_full, (uint32_t)j & 1)) bad = true;
            if (bad) sh.fail = 1;
            __syncwarp();
            tc_fence_after();
            // the partial tile to shared memory, a row per token
            for (int c0 = 0; c0 < mt; c0 += 16) {
                uint32_t v[16];
                tmem_ld16(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)c0, v);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c0 + i < mt) red[(c0 + i) * 128 + 32 * q + lane] = __uint_as_float(v[i]);
            }
            tc_fence_before();
            tile_sync(S);  // every partial of the tile is written
            // warp ew of CTA r finishes tokens r + S ew, r + S (ew + 4), ...
            if (nin) {
                const Tile t4{red, s_ga, m0, mt, rank + S * ew, lane, n, a.N, gb};
                if (S == 1) finish_tokens<F, OT, 2, 1>(a.ep, t4, bias);
                else if (S == 2) finish_tokens<F, OT, 2, 2>(a.ep, t4, bias);
                else if (S == 4) finish_tokens<F, OT, 2, 4>(a.ep, t4, bias);
                else finish_tokens<F, OT, 2, 8>(a.ep, t4, bias);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tile_sync(S);  // every partial has been read: the ring is free again
            tc_fence_after();
        }
        if (warp < 2 || warp == 6) {
            tile_sync(S);
            tile_sync(S);
            tc_fence_after();
        }
    }
    // Where a wait gave up, copies and MMAs may be under way: they complete before the
    // CTA leaves (a stage's phase also takes the arrivals of warps that gave up, so
    // this may run into its own limit).
    if ((bad || sh.fail) && warp == 0) {
        for (int k = 0; k < ns && (uint32_t)k < g; ++k) {
            int sl = r.slot - 1 - k;
            uint32_t p = r.parity;
            if (sl < 0) {
                sl += ns;
                p ^= 1u;
            }
            if (!warp_wait(&sh.full[sl], p)) bad = true;
        }
    } else if ((bad || sh.fail) && warp == 1) {
        if (elected) tc_commit(&sh.done);
        __syncwarp();  // no lane waits before the elected one has asked
        if (!warp_wait(&sh.done, 0)) bad = true;
    }
    if (bad) sh.fail = 1;
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (sh.fail && threadIdx.x == 0 && first < tiles) {
        const int chunk = first / a.tiles_p;
        e = group_of(groups, a.G, chunk, 0);
        store_out<OT>(a.ep.out, (int64_t)(groups[e].row + (chunk - groups[e].tile) * kGrpRowsTok) * a.N +
                                    (first - chunk * a.tiles_p) * 128, __int_as_float(0x7FC00000));
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kAllColumns) : "memory");
    }
}

}  // namespace lin
}  // namespace fos
