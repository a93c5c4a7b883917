// fos_linear_pair.cuh -- the product with an epilogue for many tokens: a pair
// of SMs per output tile (tcgen05 cta_group::2, M = 256).
//
// A persistent kernel of clusters of two CTAs walks 256 x 192 tiles of out.
// CTA r of a pair holds tokens 128 r .. 128 r + 127 of the tile and, of the
// weights, rows 96 r .. 96 r + 95: the pair's MMA reads each half of b from
// the SM that holds it, so an SM stages 16 KB of a and 12 KB of b for 128 x
// 192 outputs where a single SM would stage 16 + 24.  Roles of a CTA's warps:
//   warp 0     TMA producer: its halves of a and b into a ring of stages (the
//              bytes of both CTAs are counted by the full barrier of CTA 0)
//   warp 10    TMA producer of the scales, its own of a and both row tiles of
//              b, by chunks of four scale tiles along K, into a ring of its own
//   warp 1     tensor memory; in CTA 0 it issues the pair's MMAs, whose
//              completion frees the stage in both CTAs
//   warps 2-5  scales: shared memory to tensor memory (tcgen05.st), a chunk at
//              a time into a ring of three buffers, lane quadrant warp % 4; NVFP4
//              has a second group, warps 11-14, for every other chunk (one takes
//              580 cycles a chunk, more than an NVFP4 stage's MMAs)
//   warps 6-9  epilogue of the CTA's 128 tokens, lane quadrant warp % 4
// Measured, 8192 x 4096 x 14336 without an epilogue: 8 bit 284 us, 3.39 PFLOP/s
// (1.78 times the bf16 rate of a library product), at the clock that the power
// limit leaves 388 cycles a stage of four MMAs where the MMAs themselves take 384:
// bound by the tensor pipe.  NVFP4 154 us, 6.27 PFLOP/s (3.3 times): 520 cycles a
// stage of 34 KB an SM, together 17.9 TB/s out of L2, which is the bound: tiles of
// 256 x 128 (30 KB a stage, two thirds of the MMAs' time) take 436 cycles a stage,
// 180 us in all, and neither 6 instead of 3 scale buffers there nor 2 here (160 us)
// change that much.  With bias, gelu_tanh and the pre-activation kept, 8192 x
// 14336 x 4096: 311 .. 335 us in a burst, 345 .. 355 under load; 5003 x 4096 x 14336
// NVFP4 with bias, gelu and residual 107 .. 110 us, 95.5 without an epilogue.
// Tensor memory: two accumulators of 192 columns (the epilogue of a tile runs
// under the MMAs of the next) and the scale buffers of 40 columns (a: 4 per
// scale tile, b: the 6 that its 192 rows take) in the other 128.  Copying the
// scales with tcgen05.cp instead puts them into the tensor pipe itself, in
// order with the MMAs, where each 512-byte tile costs about 25 cycles and
// each batch the latency of the copy: 8192 x 4096 x 14336 took 338 us (8 bit)
// and 232 us (NVFP4) that way.
// All warps that issue asynchronous work run their loops converged and elect
// the issuing lane for the instruction alone, which keeps the operands in
// uniform registers; with a loop inside `if (lane == 0)` the issue itself was
// the bound (513 and 492 us).
// The epilogue goes by chunks of 32 tokens x 128 bytes of out.  A chunk's
// residual is fetched by TMA into the very buffer its result will leave from:
// a lane reads its 16-byte pieces, adds, and writes them back in place, so two
// buffers a warp hold the chunk in work and the last one's store or the next
// one's fetch.
#pragma once

#include "fos_linear.cuh"

namespace fos {
namespace lin {

constexpr int kPairM = 256, kPairN = 192;
constexpr int kPairABytes = 128 * kRowBytes, kPairBBytes = 96 * kRowBytes;
constexpr int kPairMaxStages = 8;
constexpr int kChunkBytes = 32 * 128;
constexpr int kPairSfCol = 2 * kPairN;

constexpr int kPairStageBytes = kPairABytes + kPairBBytes;
// A chunk of scales: four scale tiles along K of a's 128 rows and of b's two
// row tiles, one stage of F4 or four of F8.
constexpr int kSfChunkTiles = 4;
constexpr int kSfChunkA = kSfChunkTiles * kSfTileBytes, kSfChunkBytes = 3 * kSfChunkA;
// Groups of scale warps, and chunks in shared memory: a slot belongs to one
// group (the slots are a multiple of the groups), so that the waits for a slot's
// phases are all made by warps that have seen the phase before.
template <class F> constexpr int sf_groups() { return F::kGlobal ? 2 : 1; }
template <class F> constexpr int sf_slots() { return F::kGlobal ? 4 : 3; }
constexpr int kSfMaxSlots = 4;
template <class F> constexpr int pair_threads() { return 352 + 128 * (sf_groups<F>() - 1); }
// Chunks in tensor memory.  Where a chunk is a stage, no more than the ring has
// stages: the wait for the stage that used a buffer last may look back one turn of
// the ring at most, or its phase is mistaken for a later one.
constexpr int kSfBufs = 3;
constexpr int kSfCols = 16 + 24;
static_assert(kPairSfCol + kSfBufs * kSfCols <= (int)kAllColumns, "tensor memory");
template <class F> constexpr int chunk_stages() { return kSfChunkTiles / F::kSfTiles; }
// Where a chunk is a stage, the scale warps (four of each CTA) arrive at the
// stage's full barrier themselves, and a stage's empty barrier also frees its
// scale buffer: one wait and one commit a stage in the issuing warp instead of
// two, which is what binds NVFP4 (640 cycles a stage of four MMAs with two).
template <class F> constexpr bool chunk_is_stage() { return chunk_stages<F>() == 1; }

struct PairArgs {
    CUtensorMap ta;    // a codes, box 128 bytes x 128 rows
    CUtensorMap tb;    // b codes, box 128 bytes x 96 rows
    CUtensorMap tsa;   // a scales as [row tiles, kb, 512 bytes], box 1 x 4 x 512
    CUtensorMap tsb;   // b scales likewise, box 2 x 4 x 512
    CUtensorMap tout;  // out, residual, pre: box 128 bytes x 32 rows
    CUtensorMap tres;
    CUtensorMap tpre;
    Epilogue ep;
    int64_t M, N;
    int tiles_m, tiles_n;
    int band;          // tile rows of a band of the tile order
    int kb, nkb;
    int stages;
    int bufs;          // chunk buffers of an epilogue warp: 2, with pre 4
};

struct __align__(8) PairShared {
    uint64_t full[kPairMaxStages], empty[kPairMaxStages], acc_full[2], acc_empty[2], done;
    uint64_t sf_full[kSfMaxSlots], sf_empty[kSfMaxSlots], sf_ready[kSfBufs], sf_free[kSfBufs];
    uint64_t res_full[4][2];
    uint32_t tmem;
    int fail;
};

__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
// Load into this CTA's shared memory, bytes counted at `bar` (a cluster address).
__device__ __forceinline__ void pair_load_2d(void* dst, const CUtensorMap* map, int32_t x, int32_t y,
                                             uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}
// Scale tiles k ... along K of row tile r ... into this CTA.
__device__ __forceinline__ void sf_load_3d(void* dst, const CUtensorMap* map, int32_t k, int32_t r,
                                           uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(k), "r"(r), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_u32(bar)), "h"((unsigned short)3) : "memory");
}
// Arrival at a barrier of CTA 0 from either CTA of the pair, for accesses to tensor
// memory that have completed: the fences around the barrier order them (see Sync),
// so the arrival is relaxed, at the scope that holds both CTAs.
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
          "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
          "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Tile order: bands of a.band tile rows, down the rows first, so that the tiles in
// work at one time share a and b tiles in L2.
__device__ __forceinline__ void pair_tile(const PairArgs& a, int t, int32_t& m0, int32_t& n0) {
    const int per_band = a.band * a.tiles_n;
    const int band = t / per_band, r = t - band * per_band;
    const int rows = min(a.band, a.tiles_m - band * a.band);
    const int col = r / rows;
    m0 = (band * a.band + r - col * rows) * kPairM;
    n0 = col * kPairN;
}

// The biases of a tile's columns: lane l holds those of columns l, l + 32, ...
template <Out OT>
__device__ __forceinline__ void load_bias(const Epilogue& e, int64_t n0, int64_t N, int lane,
                                          float (&b)[kPairN / 32]) {
#pragma unroll
    for (int i = 0; i < kPairN / 32; ++i) {
        const int64_t n = n0 + 32 * i + lane;
        b[i] = 0.0f;
        if (n < N)
            b[i] = e.bias32 ? static_cast<const float*>(e.bias)[n] : load_out<OT>(e.bias, n);
    }
}

// 32 values as 128-bit pieces of a chunk's row: pieces p0, p0 + 1, ... of the
// 128-byte swizzle.
template <Out OT>
__device__ __forceinline__ void put_pieces(uint32_t row_addr, int lane, int p0, const float (&v)[32]) {
    constexpr int kPer = OT == Out::F32 ? 4 : 8;
#pragma unroll
    for (int k = 0; k < 32 / kPer; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (OT == Out::F32) w[i] = __float_as_uint(v[4 * k + i]);
            else w[i] = out_pair<OT>(pk(v[8 * k + 2 * i], v[8 * k + 2 * i + 1]));
        }
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         row_addr + (((p0 + k) ^ (lane & 7)) << 4)),
                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
    }
}
template <Out OT>
__device__ __forceinline__ void add_pieces(uint32_t row_addr, int lane, int p0, float (&v)[32]) {
    constexpr int kPer = OT == Out::F32 ? 4 : 8;
#pragma unroll
    for (int k = 0; k < 32 / kPer; ++k) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(row_addr + (((p0 + k) ^ (lane & 7)) << 4)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (OT == Out::F32) {
                v[4 * k + i] = fadd(v[4 * k + i], __uint_as_float(w[i]));
            } else if constexpr (OT == Out::BF16) {
                v[8 * k + 2 * i] = fadd(v[8 * k + 2 * i], __uint_as_float(w[i] << 16));
                v[8 * k + 2 * i + 1] = fadd(v[8 * k + 2 * i + 1], __uint_as_float(w[i] & 0xFFFF0000u));
            } else {
                float lo, hi;
                upk(f16x2_f32x2(w[i]), lo, hi);
                v[8 * k + 2 * i] = fadd(v[8 * k + 2 * i], lo);
                v[8 * k + 2 * i + 1] = fadd(v[8 * k + 2 * i + 1], hi);
            }
        }
    }
}

__device__ __forceinline__ void store_chunk(const CUtensorMap* map, int32_t x, int32_t y, uint32_t buf) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     map), "r"(x), "r"(y), "r"(buf) : "memory");
}

// The MMAs of a stage (one lane): nk scale tiles of it exist (F4).
template <class F>
__device__ __forceinline__ void pair_stage(uint32_t acc, uint32_t a0, uint32_t b0, uint32_t sfa,
                                           uint32_t sfb, int nk, uint32_t more) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
        if (F::kGlobal && kk >= nk) break;
        mma_issue<F, 2>(acc, a0 + 2 * kk, b0 + 2 * kk, idesc<F>(kPairM, kPairN, F::kGlobal ? 0 : kk),
                        F::kGlobal ? sfa + 4 * kk : sfa, F::kGlobal ? sfb + 6 * kk : sfb,
                        kk == 0 ? more : 1u);
    }
}

template <class F, Out OT>
__global__ void __launch_bounds__(pair_threads<F>(), 1) k_linear_pair(const __grid_constant__ PairArgs a) {
    extern __shared__ __align__(1024) unsigned char s_raw[];
    __shared__ PairShared sh;
    unsigned char* base = s_raw + ((1024u - (smem_u32(s_raw) & 1023u)) & 1023u);
    const int ns = a.stages;
    unsigned char* sA = base;
    unsigned char* sB = sA + ns * kPairABytes;
    unsigned char* sC = sB + ns * kPairBBytes;       // epilogue chunks
    static_assert(sf_slots<F>() % sf_groups<F>() == 0, "a slot belongs to one group");
    constexpr int kSfSlots = sf_slots<F>();
    unsigned char* sS = sC + 4 * a.bufs * kChunkBytes;  // scale chunks: a, then b's two row tiles
    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int rank = (int)uniform(cluster_rank());
    const int tiles = a.tiles_m * a.tiles_n;
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
            bar_init(&sh.sf_full[b], 1);
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
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are set up
    tc_fence_after();
    const uint32_t tmem = uniform(sh.tmem);
    bool bad = false;
    if (warp == 0) {
        const bool elected = elect_lane();
        const uint32_t full0 = map_rank(smem_u32(&sh.full[0]), 0);
        Ring r;
        uint32_t g = 0;
        for (int t = first; t < tiles && !bad; t += step) {
            int32_t m0, n0;
            pair_tile(a, t, m0, n0);
            const int32_t am = m0 + 128 * rank, bn = n0 + 96 * rank;
            for (int i = 0; i < a.nkb; ++i) {
                const int s = r.slot;
                if (g >= (uint32_t)ns && !warp_wait<Sync::CLUSTER>(&sh.empty[s], r.parity ^ 1u)) {
                    bad = true;
                    break;
                }
                const uint32_t bar = full0 + 8 * s;
                unsigned char *pa = sA + s * kPairABytes, *pb = sB + s * kPairBBytes;
                if (elected) {
                    if (rank == 0) mbar_expect_tx(&sh.full[s], (uint32_t)(2 * kPairStageBytes));
                    pair_load_2d(pa, &a.ta, i * kRowBytes, am, bar);
                    pair_load_2d(pb, &a.tb, i * kRowBytes, bn, bar);
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
            Ring r, f;      // stages; scale buffers
            bool here = false;  // the next stage is known to be full
            int j = 0;
            for (int t = first; t < tiles && !bad; t += step, ++j) {
                const int ab = j & 1;
                if (j >= 2 && !warp_wait<Sync::TENSOR>(&sh.acc_empty[ab], (uint32_t)((j >> 1) - 1) & 1)) {
                    bad = true;
                    break;
                }
                const uint32_t acc = tmem + (uint32_t)(ab * kPairN);
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
            int32_t m0, n0;
            pair_tile(a, t, m0, n0);
            const int32_t ra = (m0 + 128 * rank) >> 7, rb = n0 >> 7;
            for (int k = 0; k < a.kb; k += kSfChunkTiles) {
                if (chunks >= (uint32_t)kSfSlots && !warp_wait(&sh.sf_empty[f.slot], f.parity ^ 1u)) {
                    bad = true;
                    break;
                }
                unsigned char* ps = sS + f.slot * kSfChunkBytes;
                if (elected) {
                    mbar_expect_tx(&sh.sf_full[f.slot], (uint32_t)kSfChunkBytes);
                    sf_load_3d(ps, &a.tsa, k, ra, &sh.sf_full[f.slot]);
                    sf_load_3d(ps + kSfChunkA, &a.tsb, k, rb, &sh.sf_full[f.slot]);
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
    } else if (warp < 6 || warp > 10) {
        // scales: lane l of quadrant q writes row l of each 16-byte-wide tile,
        // a's four words to columns 4 kk ..., of b's eight (two row tiles) the
        // six of the tile's 192 rows to columns 16 + 6 kk ...
        const int q = warp & 3;
        const uint32_t lane_base = tmem + kPairSfCol + ((uint32_t)(32 * q) << 16);
        const uint32_t full0 = map_rank(smem_u32(&sh.full[0]), 0);
        const uint32_t ready0 = map_rank(smem_u32(&sh.sf_ready[0]), 0);
        Ring f, d;          // shared-memory slots; tensor-memory buffers
        Ring r, w;          // chunk_is_stage: its stage; the one whose buffer it takes over
        const uint32_t mine = warp < 6 ? 0u : 1u;  // the group
        uint32_t chunks = 0;
        for (int t = first; t < tiles && !bad; t += step) {
            int32_t m0, n0;
            pair_tile(a, t, m0, n0);
            const bool half = (n0 & 127) != 0;  // b starts half-way into a scale tile
            for (int i = 0; i < a.nkb; i += chunk_stages<F>()) {
                if (chunks % sf_groups<F>() != mine) {
                    if (chunks >= (uint32_t)kSfBufs) w.next(ns);
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
                    const uint4 x = *reinterpret_cast<const uint4*>(ps + kk * kSfTileBytes);
                    const uint4 u = *reinterpret_cast<const uint4*>(ps + kSfChunkA + kk * kSfTileBytes);
                    const uint4 v = *reinterpret_cast<const uint4*>(ps + 2 * kSfChunkA + kk * kSfTileBytes);
                    va[4 * kk] = x.x; va[4 * kk + 1] = x.y; va[4 * kk + 2] = x.z; va[4 * kk + 3] = x.w;
                    vb[6 * kk] = half ? u.z : u.x;
                    vb[6 * kk + 1] = half ? u.w : u.y;
                    vb[6 * kk + 2] = half ? v.x : u.z;
                    vb[6 * kk + 3] = half ? v.y : u.w;
                    vb[6 * kk + 4] = half ? v.z : v.x;
                    vb[6 * kk + 5] = half ? v.w : v.y;
                }
                if (chunks >= (uint32_t)kSfBufs) {
                    // the MMAs that read this buffer are done
                    if (chunk_is_stage<F>() ? !warp_wait<Sync::TENSOR>(&sh.empty[w.slot], w.parity)
                                            : !warp_wait<Sync::TENSOR>(&sh.sf_free[d.slot], d.parity ^ 1u)) {
                        bad = true;
                        break;
                    }
                    w.next(ns);
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
        const bool pre = a.ep.pre != nullptr, res = a.ep.residual != nullptr;
        // two slots of a buffer for out (and the residual) and, with pre, one for it
        const int slot_bytes = (pre ? 2 : 1) * kChunkBytes;
        unsigned char* bufs = sC + e * 2 * slot_bytes;
        float* s_bias = reinterpret_cast<float*>(sS + kSfSlots * kSfChunkBytes) + e * kPairN;
        const int mine = first < tiles ? (tiles - first + step - 1) / step : 0;
        const int total = mine * kChunks;
        auto fetch = [&](int c) {                       // chunk c's residual (one lane)
            int32_t m0, n0;
            pair_tile(a, first + (c / kChunks) * step, m0, n0);
            uint64_t* bar = &sh.res_full[e][c & 1];
            mbar_expect_tx(bar, kChunkBytes);
            tma_load_2d(bufs + (c & 1) * slot_bytes, &a.tres, n0 + (c % kChunks) * kCols,
                        m0 + 128 * rank + 32 * q, bar);
        };
        if (res && lane == 0 && total > 0) fetch(0);
        float bias[kPairN / 32];
        if (a.ep.bias && first < tiles) {
            int32_t m0, n0;
            pair_tile(a, first, m0, n0);
            load_bias<OT>(a.ep, n0, a.N, lane, bias);
        }
        float gb = 1.0f, ga0 = 1.0f;
        if constexpr (F::kGlobal) {
            gb = fdiv(1.0f, global_scale(a.ep.b_amax[0], a.ep.six_bound));
            if (!a.ep.a_row) ga0 = fdiv(1.0f, global_scale(a.ep.a_amax[0], a.ep.six_bound));
        }
        int c = 0, j = 0;
        for (int t = first; t < tiles; t += step, ++j) {
            int32_t m0, n0;
            pair_tile(a, t, m0, n0);
            const int32_t mw = m0 + 128 * rank + 32 * q;  // first token of this warp
            float ga = ga0;
            if constexpr (F::kGlobal)
                if (a.ep.a_row && mw + lane < a.M)
                    ga = fdiv(1.0f, global_scale(a.ep.a_amax[mw + lane], a.ep.six_bound));
            if (a.ep.bias) {  // this tile's biases to shared memory, the next one's on their way
#pragma unroll
                for (int i = 0; i < kPairN / 32; ++i) s_bias[32 * i + lane] = bias[i];
                if (t + step < tiles) {
                    int32_t mn, nn;
                    pair_tile(a, t + step, mn, nn);
                    load_bias<OT>(a.ep, nn, a.N, lane, bias);
                }
            }
            const int ab = j & 1;
            if (!bad && !warp_wait<Sync::TENSOR>(&sh.acc_full[ab], (uint32_t)(j >> 1) & 1)) bad = true;
            __syncwarp();
            tc_fence_after();
            for (int k = 0; k < kChunks; ++k, ++c) {
                const uint32_t buf = smem_u32(bufs + (c & 1) * slot_bytes);
                if (res && !bad && !warp_wait(&sh.res_full[e][c & 1], (uint32_t)(c >> 1) & 1)) bad = true;
                __syncwarp();
#pragma unroll
                for (int h = 0; h < kCols / 32; ++h) {
                    const int32_t col = k * kCols + 32 * h;
                    uint32_t u[32];
                    tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(ab * kPairN + col), u);
                    if (col + 32 == kPairN) {  // this warp has read the accumulator
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) cluster_arrive(map_rank(smem_u32(&sh.acc_empty[ab]), 0));
                    }
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        v[i] = __uint_as_float(u[i]);
                        if constexpr (F::kGlobal) v[i] = fmul(fmul(v[i], ga), gb);
                    }
                    if (a.ep.bias) {
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
                    act_apply<OT>(a.ep.act, v);
                    if (res) add_pieces<OT>(buf + lane * 128, lane, kPieces * h, v);
                    put_pieces<OT>(buf + lane * 128, lane, kPieces * h, v);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    store_chunk(&a.tout, n0 + k * kCols, mw, buf);
                    if (pre) store_chunk(&a.tpre, n0 + k * kCols, mw, buf + kChunkBytes);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    // the chunk before this one has left its slot, which the
                    // next one is fetched into and written to
                    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                    if (res && c + 1 < total) fetch(c + 1);
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
        int32_t m0, n0;
        pair_tile(a, first, m0, n0);
        if (m0 + 128 * rank < a.M)
            store_out<OT>(a.ep.out, (int64_t)(m0 + 128 * rank) * a.N + n0, __int_as_float(0x7FC00000));
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kAllColumns) : "memory");
    }
}

}  // namespace lin
}  // namespace fos
