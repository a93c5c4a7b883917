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
// scale blocks, and go from shared to tensor memory (k_linear_rows by
// tcgen05.cp, k_linear_pair through registers) in the very form the MMA reads
// them: scale j of row 32 i + l in byte j of column i of lane l, for every
// quadrant of lanes.  F4 takes one tile per MMA (its four 16-element blocks), F8
// one tile per stage, the MMA choosing byte j.
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
    static constexpr int kSfTiles = 1;    // scale tiles of a stage, per 128 rows
    static constexpr bool kGlobal = false;
};
struct F4 {
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

// What a wait orders.  CTA: memory of this CTA's own arrivals and copies.  CLUSTER:
// the same for arrivals and copies of the other CTA of a pair as well.  TENSOR:
// tensor memory alone, whichever CTA arrives: its completed accesses (wait::ld,
// wait::st, a commit) are ordered by the tcgen05 fences on both sides of the
// barrier, which itself only has to order the two threads' execution.
enum class Sync { CTA, CLUSTER, TENSOR };

#define FOS_MBAR_TEST(op, sem, hint)                                              \
    asm volatile("{\n\t.reg .pred p;\n\t"                                       \
                 "mbarrier." op ".parity" sem ".shared::cta.b64 p, [%1], %2" hint ";\n\t" \
                 "selp.u32 %0, 1, 0, p;\n\t}"                                    \
                 : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory")

// Bounded wait of a whole converged warp: every lane gets the same answer, also
// when the wait gives up.
template <Sync S = Sync::CTA>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    for (uint32_t i = 0; i < kMbarSpins; ++i) {
        uint32_t done;
        if constexpr (S == Sync::CTA) FOS_MBAR_TEST("try_wait", ".acquire.cta", ", 1000");
        else if constexpr (S == Sync::CLUSTER) FOS_MBAR_TEST("try_wait", ".acquire.cluster", ", 1000");
        else FOS_MBAR_TEST("try_wait", ".relaxed.cluster", ", 1000");
        if (__all_sync(0xFFFFFFFFu, done != 0)) return true;
    }
    return false;
}

// Whether a phase has completed, without waiting: asked a stage ahead, so that
// the answer is there when it is needed (a wait for a phase long complete
// still takes about 170 cycles, a stage's seven instructions 300).
template <Sync S = Sync::CTA>
__device__ __forceinline__ bool mbar_ask(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    if constexpr (S == Sync::CTA) FOS_MBAR_TEST("test_wait", ".acquire.cta", "");
    else if constexpr (S == Sync::CLUSTER) FOS_MBAR_TEST("test_wait", ".acquire.cluster", "");
    else FOS_MBAR_TEST("test_wait", ".relaxed.cluster", "");
    return done != 0;
}
#undef FOS_MBAR_TEST
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
__device__ __forceinline__ void sf_copy(uint32_t taddr, uint32_t lo) {
    asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
                 "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr), "r"(lo),
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
        return __uint_as_float((uint32_t)static_cast<const unsigned short*>(p)[i] << 16);
    else if constexpr (OT == Out::F16) {
        float f;
        asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(static_cast<const unsigned short*>(p)[i]));
        return f;
    } else
        return static_cast<const float*>(p)[i];
}
template <Out OT>
__device__ __forceinline__ void store_out(void* p, int64_t i, float v) {
    if constexpr (OT == Out::F32) static_cast<float*>(p)[i] = v;
    else st16(static_cast<unsigned short*>(p) + i, out_pair<OT>(pk(v, 0.0f)));
}

template <Out OT, int kN>
__device__ __forceinline__ void act_apply(int act, float (&v)[kN]) {
    constexpr bool kFine = OT == Out::F32;
    switch (static_cast<Act>(act)) {
        case Act::RELU: act_values<Act::RELU, kFine>(v); break;
        case Act::GELU: act_values<Act::GELU, kFine>(v); break;
        case Act::GELU_TANH: act_values<Act::GELU_TANH, kFine>(v); break;
        case Act::SILU:
            if constexpr (kFine) silu_values(v);
            else act_values<Act::SILU, kFine>(v);
            break;
        default: break;
    }
}

// ------------------------------------------------------------------ few tokens
// k_linear_rows: the weights are the MMA's 128 rows and the tokens its
// columns, so one token costs 16 columns of tensor work instead of 128 rows,
// and the time is that of streaming the weights.  A CTA takes 128 weight rows
// x nt <= 256 tokens; with few such tiles the K axis is split over the S CTAs
// of a cluster.  The fp32 partial tiles are laid down in shared memory, a row
// per token (over the ring of stages, idle by then): CTA r finishes tokens r,
// r + S, ..., a warp a token, each lane adding four weight rows of all S
// partials, read through the cluster's distributed shared memory in rank order
// (one fixed order of the sum), and storing them side by side.
//   warp 0    TMA producer of a stage's b tile and a tile
//   warp 6    bulk-copy producer of its scale tiles
//   warp 1    tensor memory; one elected thread copies scales and issues the MMAs
//   warps 2-5 epilogue: lane quadrant warp % 4 of the accumulator
// The scales of stage g go to ring buffer g % 4 of the tensor memory, after
// the MMAs of stage g - 4 have completed (the ring of stages is at least as
// long, so that stage's barrier is still in the phase waited for).  Every wait is
// bounded; a CTA whose wait gave up writes NaN into the first element of its
// output.
// Measured, the weights' bytes over the time against a device copy's 6.78 TB/s:
// 8 bit 14336 x 4096 (60.6 MB) 1 token 13.5 us, 4.5 TB/s (66 %); NVFP4 4096 x
// 14336 (33 MB) 48 tokens 10.9 us, 3.1 TB/s (46 %).  Of those times 4.2 .. 4.5 us
// are the launch, the first stage's way through memory and the last one's through
// the epilogue, which do not shrink with the weights; in between a CTA takes a
// stage every 0.32 us (8 bit; NVFP4 0.37), one warp issuing its four MMAs and
// scale copies.
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
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full, done;
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
__device__ __forceinline__ float4 ld_cluster4(uint32_t saddr, uint32_t rank) {
    float4 v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
                 "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(saddr), "r"(rank) : "memory");
    return v;
}
// Barrier of all threads of the S CTAs that share a tile.
__device__ __forceinline__ void tile_sync(int S) {
    __syncwarp();
    if (S > 1) cluster_sync();
    else __syncthreads();
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
            sf_copy(sfp + 4 * kk, lp + kk * kT);
#pragma unroll
            for (int q = 0; q < kQ; ++q)
                sf_copy(sfq + 4 * (kk * kQ + q), lq + (q * F::kSfTiles + kk) * kT);
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

// Four consecutive values of the output's type at element i (a multiple of 4).
template <Out OT>
__device__ __forceinline__ void load4(const void* p, int64_t i, float (&v)[4]) {
    if constexpr (OT == Out::F32) {
        const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(p) + i);
        if constexpr (OT == Out::BF16) {
            v[0] = __uint_as_float(x.x << 16); v[1] = __uint_as_float(x.x & 0xFFFF0000u);
            v[2] = __uint_as_float(x.y << 16); v[3] = __uint_as_float(x.y & 0xFFFF0000u);
        } else {
            upk(f16x2_f32x2(x.x), v[0], v[1]);
            upk(f16x2_f32x2(x.y), v[2], v[3]);
        }
    }
}
template <Out OT>
__device__ __forceinline__ void store4(void* p, int64_t i, const float* v) {
    if constexpr (OT == Out::F32) {
        const uint32_t w[4] = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                               __float_as_uint(v[3])};
        st128(static_cast<float*>(p) + i, w);
    } else {
        st64(static_cast<unsigned short*>(p) + i, out_pair<OT>(pk(v[0], v[1])),
             out_pair<OT>(pk(v[2], v[3])));
    }
}

// What a warp finishes of a tile: tokens m0 + c, c = first, first + 4 kS, ...
// below mt, at weight rows n .. n + 3.
struct Tile {
    const float* red;
    const float* ga;
    int m0, mt, first, lane;
    int64_t n, N;
    float gb;
};

// kTok tokens at a time with all of their loads in flight.
template <class F, Out OT, int kTok, int kS>
__device__ __forceinline__ void finish_tokens(const Epilogue& ep, const Tile& t,
                                              const float (&bias)[4]) {
    for (int c0 = t.first; c0 < t.mt; c0 += 4 * kS * kTok) {
        float4 p[kTok][kS];
        float rs[kTok][4], f[4 * kTok];
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            // tokens past the end repeat the last one's loads and are not stored
            const int c = min(c0 + 4 * kS * i, t.mt - 1);
            const float* at = t.red + c * 128 + 4 * t.lane;
#pragma unroll
            for (int k = 0; k < kS; ++k) {
                if constexpr (kS == 1) p[i][k] = *reinterpret_cast<const float4*>(at);
                else p[i][k] = ld_cluster4(smem_u32(at), (uint32_t)k);
            }
            if (ep.residual) load4<OT>(ep.residual, (int64_t)(t.m0 + c) * t.N + t.n, rs[i]);
        }
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const int c = c0 + 4 * kS * i;
            float4 s = p[i][0];
#pragma unroll
            for (int k = 1; k < kS; ++k) {
                s.x = fadd(s.x, p[i][k].x);
                s.y = fadd(s.y, p[i][k].y);
                s.z = fadd(s.z, p[i][k].z);
                s.w = fadd(s.w, p[i][k].w);
            }
            if constexpr (F::kGlobal) {
                const float ga = t.ga[min(c, t.mt - 1)];
                s.x = fmul(fmul(s.x, ga), t.gb);
                s.y = fmul(fmul(s.y, ga), t.gb);
                s.z = fmul(fmul(s.z, ga), t.gb);
                s.w = fmul(fmul(s.w, ga), t.gb);
            }
            f[4 * i] = fadd(s.x, bias[0]);
            f[4 * i + 1] = fadd(s.y, bias[1]);
            f[4 * i + 2] = fadd(s.z, bias[2]);
            f[4 * i + 3] = fadd(s.w, bias[3]);
            if (ep.pre && c < t.mt) store4<OT>(ep.pre, (int64_t)(t.m0 + c) * t.N + t.n, f + 4 * i);
        }
        act_apply<OT>(ep.act, f);
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const int c = c0 + 4 * kS * i;
            if (ep.residual) {
#pragma unroll
                for (int x = 0; x < 4; ++x) f[4 * i + x] = fadd(f[4 * i + x], rs[i][x]);
            }
            if (c < t.mt) store4<OT>(ep.out, (int64_t)(t.m0 + c) * t.N + t.n, f + 4 * i);
        }
    }
}

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
            bar_init(&sh.done, 1);
            sh.fail = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // everything that needs no data of the kernel before comes before the wait
    // for it (that kernel is still running: six stages leave room for this CTA)
    const bool elected = elect_lane();
    uint32_t g = 0;   // stages loaded (warps 0, 6) or consumed (warp 1) so far
    Ring r, w;        // the stage in work; warp 1: the one whose scales are overwritten
    bool bad = false;
    bool here = false, free = false;  // warp 1: the next stage is full, its scale buffer is free
    int j = 0;        // tiles of this CTA so far
    int tq = first / a.tiles_p, tp = first - tq * a.tiles_p;
    __syncwarp();
    __syncthreads();
    chain_wait();
    chain_release();
    uint32_t tmem = 0;
    if (warp != 0 && warp != 6) {  // the producers need no tensor memory
        if (warp == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(&sh.tmem)), "r"(kAllColumns) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
        tc_fence_before();
        __syncwarp();
        asm volatile("bar.sync 1, 160;" ::: "memory");
        tc_fence_after();
        tmem = uniform(sh.tmem);
    }
    for (int t = first; t < a.tiles; t += step, ++j) {
        if (j > 0) {
            tq = t / a.tiles_p;
            tp = t - tq * a.tiles_p;
        }
        const int n0 = tp * 128, m0 = tq * nt;
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
            const int q = warp & 3, e = warp - 2;
            const int mt = min(nt, (int)a.M - m0);
            // finishing, lane l has weight rows 4 l .. 4 l + 3 of the tile
            const int64_t n = n0 + 4 * lane;
            const bool nin = n < a.N;
            float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (a.ep.bias && nin) {
                if (a.ep.bias32) load4<Out::F32>(a.ep.bias, n, bias);
                else load4<OT>(a.ep.bias, n, bias);
            }
            float gb = 1.0f;
            if constexpr (F::kGlobal) {
                // the tokens' decode scales, once per tile
                gb = fdiv(1.0f, global_scale(a.ep.b_amax[0], a.ep.six_bound));
                for (int c = 32 * e + lane; c < mt; c += 128)
                    s_ga[c] = fdiv(1.0f, global_scale(a.ep.a_amax[a.ep.a_row ? m0 + c : 0],
                                                      a.ep.six_bound));
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
            // warp e of CTA r finishes tokens r + S e, r + S (e + 4), ...
            if (nin) {
                const Tile t4{red, s_ga, m0, mt, rank + S * e, lane, n, a.N, gb};
                if (S == 1) finish_tokens<F, OT, 4, 1>(a.ep, t4, bias);
                else if (S == 2) finish_tokens<F, OT, 4, 2>(a.ep, t4, bias);
                else if (S == 8) finish_tokens<F, OT, 2, 8>(a.ep, t4, bias);
                // (4096 x 14336 NVFP4: 16 tokens 9.8 us two at a time, 10.4 four at
                // a time; 48 tokens 11.5 and 11.0)
                else if (mt <= 32) finish_tokens<F, OT, 2, 4>(a.ep, t4, bias);
                else finish_tokens<F, OT, 4, 4>(a.ep, t4, bias);
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
    // Every copy and MMA issued has completed before the CTA leaves: the epilogue
    // has seen each tile's accumulator full, so there is something to wait for
    // only where a wait gave up.
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
