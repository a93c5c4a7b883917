// fos_linear.cuh -- products of quantized operands with an epilogue, on the
// 5th-generation tensor cores of sm_103a (tcgen05):
//
//   v[m][n]   = (a . b^T)[m][n] * g_a(m) * g_b + bias[n]
//   pre[m][n] = v                         (optional)
//   out[m][n] = act(v) + residual[m][n]
//
// a [M, K] are tokens, b [N, K] weights.  Formats (struct F8, F4): E4M3 codes
// with a UE8M0 scale per 32 elements (kind::mxf8f6f4, scale_vec::1X; the g are
// 1), or E2M1 codes with an E4M3 scale per 16 (kind::mxf4nvf4, scale_vec::4X;
// g the global decode scales).  Both keep 128 code bytes of a row per K stage
// (the 128-byte swizzle) and take four MMAs of 32 bytes each; their scales
// come as the 512-byte tiles of the tiled layout, one tile per 128 rows and 4
// scale blocks, copied from shared to tensor memory by tcgen05.cp in the very
// form the MMA reads them: scale j of row 32 i + l in byte j of column i of
// lane l, for every quadrant of lanes.  F4 takes one tile per MMA (its four
// 16-element blocks), F8 one tile per stage, the MMA choosing byte j.
#pragma once

#include <cuda.h>

#include "fos_act.cuh"
#include "fos_kernels.cuh"
#include "fos_mma.cuh"

namespace fos {
namespace lin {

using mma::bar_arrive;
using mma::bar_init;
using mma::bulk_load;
using mma::tc_commit;
using mma::tc_fence_after;
using mma::tc_fence_before;

}  // namespace lin

// Everything the epilogue needs.
struct Epilogue {
    const void* bias;      // [N], fp32 or the output's type, or null
    const void* residual;  // [M, N], the output's type, or null
    void* pre;             // [M, N], the output's type, or null
    void* out;
    const float* a_amax;   // F4: [1] or [M]
    const float* b_amax;   // F4: [1]
    int a_row;             // F4: a_amax per row
    int act;
    int bias32;
    float six_bound;
};

// One product, as the host passes it to the launchers.
struct LinearCall {
    const uint8_t *a, *as, *b, *bs;  // codes and tiled scales
    int64_t M, N, K;
    Epilogue ep;
    In out;                          // type of out, residual and pre
    bool fmt4;
};

namespace lin {

struct F8 {
    static constexpr int kStageK = 128;   // K elements of a stage
    static constexpr int kSfTiles = 1;    // scale tiles of a stage, per 128 rows
    static constexpr bool kGlobal = false;
};
struct F4 {
    static constexpr int kStageK = 256;
    static constexpr int kSfTiles = 4;
    static constexpr bool kGlobal = true;
};
constexpr int kRowBytes = 128;      // code bytes of a row per stage
constexpr int kSfTileBytes = 512;

// Instruction descriptor: element formats (E4M3 0, E2M1 1 or in the F8 kind
// E4M3 0) in bits 7-9 and 10-12, N >> 3 in 17-22, scale type in 23 (UE8M0 1),
// M >> 4 in 24-28, scale bytes of b and a in 4-5 and 29-30.
template <class F>
__device__ __forceinline__ uint32_t idesc(int m, int n, int sf_id) {
    const uint32_t fmt = F::kGlobal ? (1u << 7) | (1u << 10) : (1u << 23);
    return fmt | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24) |
           ((uint32_t)sf_id << 4) | ((uint32_t)sf_id << 29);
}

// Bounded wait of a whole converged warp: every lane gets the same answer, also
// when the wait gives up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    for (uint32_t i = 0; i < kMbarSpins; ++i) {
        uint32_t done;
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
        if (__all_sync(0xFFFFFFFFu, done != 0)) return true;
    }
    return false;
}

// Whether a phase has completed, without waiting: asked a stage ahead, so that
// the answer is there when it is needed (a wait for a phase long complete
// still takes about 170 cycles, a stage's seven instructions 300).
__device__ __forceinline__ bool mbar_ask(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return done != 0;
}
// Lane 0's value for the whole warp: the compiler then knows it is uniform and
// keeps what follows from it (addresses, descriptors, loop counts) in uniform
// registers, which the tensor instructions read.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }
__device__ __forceinline__ bool warp_agrees(bool v) { return __all_sync(0xFFFFFFFFu, v); }

// One lane of the warp, the same one each time: the warp's loops run converged
// (their values stay in uniform registers, where the tensor instructions take
// their operands from) and only the issue itself is one lane's.
__device__ __forceinline__ bool elect_lane() {
    uint32_t p;
    __syncwarp();  // a diverged warp would elect a lane in each part
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(p));
    return p != 0;
}

// Descriptors are a constant high word and a low word that holds the address;
// moving by b bytes adds b / 16 to the low word.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // of desc_sw128
constexpr uint32_t kSfDescHi = (128u >> 4) | (1u << 14);               // of a scale tile
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) {
    return ((saddr & 0x3FFFFu) >> 4) | (1u << 16);
}
__device__ __forceinline__ uint32_t sf_desc_lo(uint32_t saddr) {
    return ((saddr & 0x3FFFFu) >> 4) | ((128u >> 4) << 16);
}

#define FOS_MMA_TEXT(group, kind)                                                              \
    "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %6, 0;\n\t"                      \
    "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"                                        \
    "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], a, b, %3, [%4], [%5], p;\n\t}"

// One MMA: accumulator, low descriptor words of both operands, instruction
// descriptor, scale columns.
template <class F, int kPair>
__device__ __forceinline__ void mma_issue(uint32_t acc, uint32_t alo, uint32_t blo, uint32_t id,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if constexpr (F::kGlobal && kPair == 1)
        asm volatile(FOS_MMA_TEXT("1", "mxf4nvf4.block_scale.scale_vec::4X") ::"r"(acc), "r"(alo),
                     "r"(blo), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(kDescHi) : "memory");
    else if constexpr (F::kGlobal)
        asm volatile(FOS_MMA_TEXT("2", "mxf4nvf4.block_scale.scale_vec::4X") ::"r"(acc), "r"(alo),
                     "r"(blo), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(kDescHi) : "memory");
    else if constexpr (kPair == 1)
        asm volatile(FOS_MMA_TEXT("1", "mxf8f6f4.block_scale.scale_vec::1X") ::"r"(acc), "r"(alo),
                     "r"(blo), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(kDescHi) : "memory");
    else
        asm volatile(FOS_MMA_TEXT("2", "mxf8f6f4.block_scale.scale_vec::1X") ::"r"(acc), "r"(alo),
                     "r"(blo), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(kDescHi) : "memory");
}
#undef FOS_MMA_TEXT

// One scale tile from shared (low descriptor word) to tensor memory.
template <int kPair>
__device__ __forceinline__ void sf_copy(uint32_t taddr, uint32_t lo) {
    if constexpr (kPair == 1)
        asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
                     "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr), "r"(lo),
                     "r"(kSfDescHi) : "memory");
    else
        asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
                     "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr), "r"(lo),
                     "r"(kSfDescHi) : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

template <Out OT>
__device__ __forceinline__ float load_out(const void* p, int64_t i) {
    if constexpr (OT == Out::BF16)
        return __uint_as_float((uint32_t)__ldg(static_cast<const unsigned short*>(p) + i) << 16);
    else if constexpr (OT == Out::F16) {
        float f;
        asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(__ldg(static_cast<const unsigned short*>(p) + i)));
        return f;
    } else
        return __ldg(static_cast<const float*>(p) + i);
}
template <Out OT>
__device__ __forceinline__ void store_out(void* p, int64_t i, float v) {
    if constexpr (OT == Out::F32) static_cast<float*>(p)[i] = v;
    else st16(static_cast<unsigned short*>(p) + i, out_pair<OT>(pk(v, 0.0f)));
}

template <int kN>
__device__ __forceinline__ void act_apply(int act, float (&v)[kN]) {
    switch (static_cast<Act>(act)) {
        case Act::RELU: act_values<Act::RELU>(v); break;
        case Act::GELU: act_values<Act::GELU>(v); break;
        case Act::GELU_TANH: act_values<Act::GELU_TANH>(v); break;
        case Act::SILU: act_values<Act::SILU>(v); break;
        default: break;
    }
}

// ------------------------------------------------------------------ few tokens
// k_linear_rows: the weights are the MMA's 128 rows and the tokens its
// columns, so one token costs 16 columns of tensor work instead of 128 rows,
// and the time is that of streaming the weights.  A CTA takes 128 weight rows
// x nt <= 256 tokens; with few such tiles the K axis is split over the S CTAs
// of a cluster, whose fp32 partial tiles meet in shared memory: CTA r adds
// tokens r, r + S, ... of all S partials, read through the cluster's
// distributed shared memory in rank order (one fixed order of the sum).
//   warp 0    TMA producer of a stage's b tile and a tile
//   warp 6    bulk-copy producer of its scale tiles
//   warp 1    tensor memory; one thread copies scales and issues the MMAs
//   warps 2-5 epilogue: lane quadrant warp % 4 of the accumulator
// The scales of stage g go to ring buffer g % 4 of the tensor memory, after
// the MMAs of stage g - 4 have completed (the ring of stages is at least as
// long, so that stage's barrier is still in the phase waited for).  Every wait is bounded; a CTA whose
// wait gave up writes NaN into the first element of its output.
struct RowsArgs {
    CUtensorMap tp;      // b codes, box 128 bytes x 128 rows
    CUtensorMap tq;      // a codes, box 128 bytes x nt rows
    const uint8_t* sfp;  // b scales, tiled
    const uint8_t* sfq;  // a scales, tiled
    Epilogue ep;
    int64_t M, N;
    int tiles;           // tiles_p * tiles_q
    int kb;              // scale tiles along K (4 blocks each)
    int nkb;             // stages along K
    int tiles_p;
    int nt;              // tokens per tile (multiple of 16)
    int splits;          // cluster size
    int stages;
};

constexpr int kRowsThreads = 224;
constexpr int kMaxStages = 6;  // measured against 4, 5, 8 and 12: the fastest over 1 to 64 tokens
constexpr int kSfRing = 4;
constexpr uint32_t kAllColumns = 512;

struct __align__(8) RowsShared {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full, acc_empty, done;
    uint32_t tmem;
    int fail;
};

template <class F>
__host__ __device__ constexpr int rows_q_atoms(int nt) { return (nt + 127) / 128; }
// Bytes of one stage: codes of both operands, scale tiles of both.
template <class F>
__host__ __device__ constexpr int rows_stage_bytes(int nt) {
    return (128 + nt) * kRowBytes + (1 + rows_q_atoms<F>(nt)) * F::kSfTiles * kSfTileBytes;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t saddr, uint32_t rank) {
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
                 "ld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v) : "r"(saddr), "r"(rank) : "memory");
    return v;
}

// Position in a ring of n slots: slot and the parity of its current use.
struct Ring {
    int slot = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next(int n) {
        if (++slot == n) {
            slot = 0;
            parity ^= 1u;
        }
    }
};

// The scale copies and MMAs of one stage (one lane): kQ scale tiles of tokens
// per weight scale tile, nk scale tiles along K.
template <class F, int kQ>
__device__ __forceinline__ void rows_stage(uint32_t acc, uint32_t p0, uint32_t q0, uint32_t id,
                                           uint32_t sfp, uint32_t sfq, uint32_t lp, uint32_t lq,
                                           int nk, uint32_t more) {
    constexpr uint32_t kT = kSfTileBytes >> 4;
#pragma unroll
    for (int kk = 0; kk < F::kSfTiles; ++kk) {
        if (kk < nk) {
            sf_copy<1>(sfp + 4 * kk, lp + kk * kT);
#pragma unroll
            for (int q = 0; q < kQ; ++q)
                sf_copy<1>(sfq + 4 * (kk * kQ + q), lq + (q * F::kSfTiles + kk) * kT);
        }
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
        if (F::kGlobal && kk >= nk) break;
        mma_issue<F, 1>(acc, p0 + 2 * kk, q0 + 2 * kk,
                        F::kGlobal ? id : id | ((uint32_t)kk << 4) | ((uint32_t)kk << 29),
                        F::kGlobal ? sfp + 4 * kk : sfp, F::kGlobal ? sfq + 4 * kk * kQ : sfq,
                        kk == 0 ? more : 1u);
    }
}

// The residuals of kN tokens from `at` on, dat apart (the first cnt of them).
template <Out OT, int kN>
__device__ __forceinline__ void load_residual(const Epilogue& e, int64_t at, int64_t dat, int cnt,
                                              float (&r)[kN]) {
#pragma unroll
    for (int i = 0; i < kN; ++i) r[i] = e.residual && i < cnt ? load_out<OT>(e.residual, at + i * dat) : 0.0f;
}

// The epilogue of kN tokens of one weight row, their scaled sums in v: stores
// at `at`, dat apart (the first cnt of them).
template <Out OT, int kN>
__device__ __forceinline__ void finish_rows(const Epilogue& e, float (&v)[kN], const float (&r)[kN],
                                            int64_t at, int64_t dat, int cnt, float bias) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = fadd(v[i], bias);
    if (e.pre) {
#pragma unroll
        for (int i = 0; i < kN; ++i)
            if (i < cnt) store_out<OT>(e.pre, at + i * dat, v[i]);
    }
    act_apply(e.act, v);
    if (e.residual) {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = fadd(v[i], r[i]);
    }
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if (i < cnt) store_out<OT>(e.out, at + i * dat, v[i]);
}

// Barrier of the four epilogue warps.
__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <class F, Out OT>
__global__ void __launch_bounds__(kRowsThreads, 1) k_linear_rows(const __grid_constant__ RowsArgs a) {
    extern __shared__ __align__(1024) unsigned char s_raw[];
    __shared__ RowsShared sh;
    __shared__ float s_ga[F::kGlobal ? 256 : 1];  // the tokens' decode scales
    unsigned char* base = s_raw + ((1024u - (smem_u32(s_raw) & 1023u)) & 1023u);
    const int nt = a.nt, S = a.splits, qa = rows_q_atoms<F>(nt), ns = a.stages;
    const int qbytes = nt * kRowBytes;
    constexpr int kPBytes = 128 * kRowBytes, kSfP = F::kSfTiles * kSfTileBytes;
    unsigned char* sP = base;
    unsigned char* sQ = sP + ns * kPBytes;
    unsigned char* sFP = sQ + ns * qbytes;
    unsigned char* sFQ = sFP + ns * kSfP;
    float* red = reinterpret_cast<float*>(base);  // [nt][128] partial tile, over the ring
    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int rank = S > 1 ? (int)uniform(cluster_rank()) : 0;
    const int first = (int)blockIdx.x / S, step = (int)gridDim.x / S;
    // this CTA's stages of every tile
    const int k_lo = a.nkb * rank / S, k_hi = a.nkb * (rank + 1) / S;
    if (warp == 0) {
        if (lane < ns) {
            bar_init(&sh.full[lane], 2);
            bar_init(&sh.empty[lane], 1);
        } else if (lane == 31) {
            bar_init(&sh.acc_full, 1);
            bar_init(&sh.acc_empty, 4);
            bar_init(&sh.done, 1);
            sh.fail = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    chain_wait();
    chain_release();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh.tmem)), "r"(kAllColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(sh.tmem);
    uint32_t g = 0;   // stages loaded (warps 0, 6) or consumed (warp 1) so far
    Ring r, w;        // the stage in work; warp 1: the one whose scales are overwritten
    const bool elected = elect_lane();
    bool bad = false;
    bool here = false, free = false;  // warp 1: the next stage is full, its scale buffer is free
    int j = 0;        // tiles of this CTA so far
    for (int t = first; t < a.tiles; t += step, ++j) {
        const int tq = t / a.tiles_p;
        const int n0 = (t - tq * a.tiles_p) * 128, m0 = tq * nt;
        if (warp == 0) {
            for (int i = k_lo; i < k_hi && !bad; ++i) {
                const int s = r.slot;
                if (g >= (uint32_t)ns && !warp_wait(&sh.empty[s], r.parity ^ 1u)) {
                    bad = true;
                    break;
                }
                unsigned char *dp = sP + s * kPBytes, *dq = sQ + s * qbytes;
                if (elected) {
                    mbar_expect_tx(&sh.full[s], (uint32_t)(kPBytes + qbytes));
                    tma_load_2d(dp, &a.tp, i * kRowBytes, n0, &sh.full[s]);
                    tma_load_2d(dq, &a.tq, i * kRowBytes, m0, &sh.full[s]);
                }
                __syncwarp();
                ++g;
                r.next(ns);
            }
        } else if (warp == 6) {
            const uint8_t* pp = a.sfp + ((int64_t)(n0 >> 7) * a.kb + F::kSfTiles * k_lo) * kSfTileBytes;
            // token tiles past the end of a have no scale tile: any finite
            // scales do (their codes are zeros)
            const int last = (int)((a.M + 127) >> 7) - 1, q0 = m0 >> 7;
            const uint8_t* pq0 = a.sfq + ((int64_t)q0 * a.kb + F::kSfTiles * k_lo) * kSfTileBytes;
            const uint8_t* pq1 = a.sfq + ((int64_t)min(q0 + 1, last) * a.kb + F::kSfTiles * k_lo) * kSfTileBytes;
            for (int i = k_lo; i < k_hi && !bad; ++i) {
                const int s = r.slot;
                if (g >= (uint32_t)ns && !warp_wait(&sh.empty[s], r.parity ^ 1u)) {
                    bad = true;
                    break;
                }
                const uint32_t bytes = (uint32_t)(min(F::kSfTiles, a.kb - F::kSfTiles * i) * kSfTileBytes);
                unsigned char *dp = sFP + s * kSfP, *dq = sFQ + s * qa * kSfP;
                if (elected) {
                    mbar_expect_tx(&sh.full[s], (1 + qa) * bytes);
                    bulk_load(dp, pp, bytes, &sh.full[s]);
                    bulk_load(dq, pq0, bytes, &sh.full[s]);
                    if (qa == 2) bulk_load(dq + kSfP, pq1, bytes, &sh.full[s]);
                }
                __syncwarp();
                pp += kSfP;
                pq0 += kSfP;
                pq1 += kSfP;
                ++g;
                r.next(ns);
            }
        } else if (warp == 1) {
            if (!bad && j >= 1 && S == 1 && !warp_wait(&sh.acc_empty, (uint32_t)(j - 1) & 1)) bad = true;
            tc_fence_after();
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
                const uint32_t lp = sf_desc_lo(smem_u32(sFP) + s * kSfP);
                const uint32_t lq = sf_desc_lo(smem_u32(sFQ) + s * qa * kSfP);
                const uint32_t p0 = desc_lo(smem_u32(sP) + s * kPBytes);
                const uint32_t q0 = desc_lo(smem_u32(sQ) + s * qbytes);
                const uint32_t id = idesc<F>(128, nt, 0);
                const uint32_t more = i > k_lo;
                if (elected) {
                    if (qa == 1) rows_stage<F, 1>(tmem, p0, q0, id, sfp, sfq, lp, lq, nk, more);
                    else rows_stage<F, 2>(tmem, p0, q0, id, sfp, sfq, lp, lq, nk, more);
                    tc_commit(&sh.empty[s]);
                }
                __syncwarp();
                ++g;
            }
            if (!bad && elected) tc_commit(&sh.acc_full);
            __syncwarp();
        } else {
            const int q = warp & 3;
            const int nl = 32 * q + lane;            // weight row of the tile
            const int64_t n = n0 + nl;
            const int mt = min(nt, (int)a.M - m0);
            const bool nin = n < a.N;
            float bias = 0.0f;
            if (a.ep.bias && nin)
                bias = a.ep.bias32 ? __ldg(static_cast<const float*>(a.ep.bias) + n)
                                   : load_out<OT>(a.ep.bias, n);
            float gb = 1.0f;
            if constexpr (F::kGlobal) {
                // the tokens' decode scales, once per tile
                gb = fdiv(1.0f, global_scale(a.ep.b_amax[0], a.ep.six_bound));
                epilogue_sync();  // the tile before has read its own
                for (int c = nl; c < mt; c += 128)
                    s_ga[c] = fdiv(1.0f, global_scale(__ldg(a.ep.a_amax + (a.ep.a_row ? m0 + c : 0)),
                                                      a.ep.six_bound));
                epilogue_sync();
            }
            if (!bad && !warp_wait(&sh.acc_full, (uint32_t)j & 1)) bad = true;
            __syncwarp();
            tc_fence_after();
            const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16);
            if (S > 1) {
                for (int c0 = 0; c0 < mt; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld16(lane_base + (uint32_t)c0, v);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c0 + i < mt) red[(c0 + i) * 128 + nl] = __uint_as_float(v[i]);
                }
                tc_fence_before();
                __syncwarp();
                cluster_sync();  // every partial of the tile is written
                if (nin) {
                    // four tokens at a time, all of their loads in flight
                    for (int c = rank; c < mt; c += 4 * S) {
                        const int cnt = (mt - c + S - 1) / S;
                        const int64_t at = (int64_t)(m0 + c) * a.N + n, dat = (int64_t)S * a.N;
                        float f[4], rs[4], p[4][8];
                        load_residual<OT>(a.ep, at, dat, cnt, rs);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (k < S && i < cnt)
                                    p[i][k] = ld_cluster(smem_u32(red + (c + i * S) * 128 + nl), (uint32_t)k);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            f[i] = p[i][0];
#pragma unroll
                            for (int k = 1; k < 8; ++k)
                                if (k < S) f[i] = fadd(f[i], p[i][k]);
                            if constexpr (F::kGlobal)
                                f[i] = fmul(fmul(f[i], s_ga[i < cnt ? c + i * S : c]), gb);
                        }
                        finish_rows<OT>(a.ep, f, rs, at, dat, cnt, bias);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                cluster_sync();  // every partial has been read: the ring is free again
            } else {
                for (int c0 = 0; c0 < mt; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld16(lane_base + (uint32_t)c0, v);
                    if (nin) {
                        const int64_t at = (int64_t)(m0 + c0) * a.N + n;
                        float f[16], rs[16];
                        load_residual<OT>(a.ep, at, a.N, mt - c0, rs);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            f[i] = __uint_as_float(v[i]);
                            if constexpr (F::kGlobal)
                                f[i] = fmul(fmul(f[i], s_ga[min(c0 + i, mt - 1)]), gb);
                        }
                        finish_rows<OT>(a.ep, f, rs, at, a.N, mt - c0, bias);
                    }
                    __syncwarp();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&sh.acc_empty);
                __syncwarp();
            }
        }
        if (S > 1 && (warp < 2 || warp == 6)) {
            __syncwarp();
            cluster_sync();
            cluster_sync();
            tc_fence_after();
        }
    }
    // drain: every copy and MMA issued has completed before the CTA leaves
    if (warp == 0) {
        for (int k = 0; k < ns && (uint32_t)k < g; ++k) {
            int sl = r.slot - 1 - k;
            uint32_t p = r.parity;
            if (sl < 0) {
                sl += ns;
                p ^= 1u;
            }
            if (!warp_wait(&sh.full[sl], p)) bad = true;
        }
    } else if (warp == 1) {
        if (elected) tc_commit(&sh.done);
        __syncwarp();  // no lane waits before the elected one has asked
        if (!warp_wait(&sh.done, 0)) bad = true;
    }
    if (bad) sh.fail = 1;
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (sh.fail && threadIdx.x == 0 && first < a.tiles)
        store_out<OT>(a.ep.out, (int64_t)(first / a.tiles_p) * nt * a.N + (first % a.tiles_p) * 128,
                      __int_as_float(0x7FC00000));
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kAllColumns) : "memory");
    }
}

}  // namespace lin
}  // namespace fos
