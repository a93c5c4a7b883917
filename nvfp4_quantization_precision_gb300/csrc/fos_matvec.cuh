// fos_matvec.cuh -- few rows of 16 or 32 bits times NVFP4 weights:
//
//   out[p][n] = act(g[e] sum_k x[p / rep][k] w[e][n][k] + bias[e][n]) + residual[p][n]
//
// e = ids[p] (0 without ids), w = e2m1(code) * e4m3(scale of its 16 elements) and
// g[e] the weight's global decode scale.  No element of x is rounded before the sum,
// whatever stands beside it.  Bound by the weights' bytes (9/16 byte an element), close
// behind by the instructions that unpack them.
//
// A weight w is exact in fp16 (two significant bits times four, 2^-10 to 2688), so the
// sums are formed by mma.m16n8k16 with weights as the 16 rows, rows of x as the 8
// columns and fp32 accumulators.  tcgen05 would take its operands through shared or
// tensor memory, two more moves of every unpacked weight, for tiles of 128 rows that
// eight columns never fill.
//   unpack   two weights by one conversion from E2M1, times the pair's scale: 16.4 cycles
//            of an SM's quarter for the 256 weights of a warp's word, 10.4 of them the MMA's (by
//            masks and shifts 28.3, whose ALU takes 2 cycles an instruction: 16.8 us
//            instead of 11.7 for one row x 14336 x 4096).
//   order    a lane takes 32 elements of a row (16 bytes) and gives them to eight
//            MMAs, four a time: any order of k serves as long as x has the same.
//   x        is brought to fp16 in shared memory once a CTA (put_x below): bf16 times a power
//            of two, fp32 in three pieces of 11 significant bits, which take three
//            columns, two rows at a time.  Elements too small beside the largest of their
//            128 are left and take turns of their own.
// A CTA takes 16 kR weight rows, kR of 1 .. 4 chosen so that the CTAs fill the device
// evenly.  Its eight warps split K by steps of 128, each with a ring of its own of
// ring<kR>() steps' codes, filled by TMA (zeros past K), and with few CTAs the CTAs of a
// cluster split K too; partial sums are added in one fixed order, warps first.
// Measured, GPU time in a graph: one row x 14336 x 4096 (33 MB), bias and silu 11.9 us, 2.8
// TB/s, of which about 4 us are the launch, x's way to shared memory and the sums; eight
// rows of six experts x 4096 x 14336 (198 MB) 48.6 us, 4.1 TB/s.  The copies alone take 6.4 and 31
// us, unpacking and MMAs alone 6.2 and 30: with four warps a scheduler they overlap only
// in part.  Measured and not kept: shares of row tiles walked by as many CTAs as fit, the
// ring running ahead over their ends, 54 us; 256 elements a step 68; rings as deep as
// shared memory allows 13.2 and 49; one ring a CTA 12.2 and 61.
// With ids, grid row p handles the rows of expert ids[p] at once if p is the first
// of them (the weights are read once), else nothing.
#pragma once

#include "fos_groups.cuh"
#include "fos_linear.cuh"

namespace fos {

struct MatvecArgs {
    CUtensorMap codes;      // [G * N, K / 2], box 16 kR rows x 64 bytes
    const uint8_t* b;       // the codes themselves
    const void* x;          // [M / rep, K]
    const int32_t* ids;     // [M] or null
    const uint8_t* scales;  // [G] x tiled
    Epilogue ep;            // b_amax [G]
    int64_t scale_bytes;    // of one expert
    int M, N, K, G, rep;
    int kt;                 // scale tiles along K (64 elements)
    int splits;
    int out_dt;             // Out
};

namespace matvec {

constexpr int kWarpsMv = 8, kStepK = 128, kMaxRows = 1024;
constexpr int kStepBytes = kStepK / 2;  // of a row of codes
template <int kR> constexpr int ring() { return kR < 4 ? 3 : 2; }  // steps of a warp: two CTAs an SM
// Floats of a column of partial sums: a multiple of 16, but not of 32, plus 4, so that a
// warp's stores touch every bank once.
template <int kR> constexpr int line() { return 16 * kR + (kR % 2 ? 20 : 4); }
template <int kR> constexpr int ring_bytes() { return kWarpsMv * ring<kR>() * 16 * kR * kStepBytes; }
// x in fp16: kXBytes of columns and steps, a step of zeros, and each row's factor of a step.
constexpr int kXStep = kStepK * 2, kXSteps = 128, kXBytes = kXSteps * kXStep;
template <int kR> constexpr int smem_bytes() { return ring_bytes<kR>() + kXBytes + 64 + kXSteps * 4; }

template <In XT> constexpr int tokens() { return XT == In::F32 ? 2 : 8; }

__device__ __forceinline__ uint32_t mul_pair(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// The eight weights of a word of codes as pairs of neighbours, times the scale pair.
__device__ __forceinline__ void unpack(uint32_t w, uint32_t s, uint32_t (&v)[4]) {
    asm("{\n\t.reg .b8 q0, q1, q2, q3;\n\tmov.b32 {q0, q1, q2, q3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, q0;\n\tcvt.rn.f16x2.e2m1x2 %1, q1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, q2;\n\tcvt.rn.f16x2.e2m1x2 %3, q3;\n\t}"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul_pair(v[i], s);
}
// Two scales' E4M3 bytes (low half of `two`) as a pair.
__device__ __forceinline__ uint32_t scale_pair(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                      uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// A lane's products of a step's 16 weight rows (32 codes of rows g and g + 8, their two
// scales each) with its column of x.
__device__ __forceinline__ void mma_tile(float (&sum)[4], uint4 lo4, uint4 hi4, uint32_t s0, uint32_t s1,
                                         const uint4 (&f)[4]) {
    const uint32_t w0[4] = {lo4.x, lo4.y, lo4.z, lo4.w}, w1[4] = {hi4.x, hi4.y, hi4.z, hi4.w};
    const uint32_t p0 = scale_pair(s0), p1 = scale_pair(s1);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t u[4], v[4];
        unpack(w0[q], __byte_perm(p0, 0u, q < 2 ? 0x1010 : 0x3232), u);
        unpack(w1[q], __byte_perm(p1, 0u, q < 2 ? 0x1010 : 0x3232), v);
        mma16(sum, u[0], v[0], u[1], v[1], f[q].x, f[q].y);
        mma16(sum, u[2], v[2], u[3], v[3], f[q].z, f[q].w);
    }
}
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint4 ld128(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ld_u16(const void* p) {
    uint32_t v;
    asm volatile("{\n\t.reg .b16 h;\n\tld.global.b16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.volatile.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t* v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}

// Where the 16-byte piece q (0 .. 3) of lane t's 32 elements of a column's step lies in
// its 256 bytes: the four lanes of two neighbouring columns touch every bank once.
__device__ __forceinline__ uint32_t x_piece(int t, int col, int q) {
    return (uint32_t)((t >> 1) * 128 + ((((t & 1) * 4 + q) ^ ((t >> 1) + 2 * (col & 1))) << 4));
}

__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// How x comes to fp16 without a loss.  A row's 128 elements of a step are multiplied by
// the power of two that brings the largest finite one to 2^14 .. 2^15.  bf16: fp16, whose
// last place is 2^-24 at least, then holds every element down to 2^-31 of it (by their
// exponents) exactly.  fp32: three pieces of 11 significant bits, each the rounding of
// what is left, the second times 2^11, the third times 2^22; with a last place of 2^-46
// they hold every element down to 2^-37.  Elements below that are left, zeros in their
// place, and their products are added in turns of their own (add_left), in each of which
// the largest of those left sets the power, until none is: nine at most for the whole
// range of either type.  (The large elements cannot decide how the small ones are held:
// where they meet zero weights the sum is of the small ones alone.)  Looking for them
// costs up to 0.4 us a call (1024 x 1024 3.4 us without, 3.8 with; 2048 x 7168 6.2 .. 6.5 and
// 6.5 .. 6.8; ten fp32 rows x 3520 x 6784 33.8 and 35.3; 14336 x 4096 11.5 and 11.3, a product
// less a sum).  With the turns in the loop over steps 14336 x 4096 took 11.9; with
// infinities and NaN looked for in every block 1408 x 2048 of 16 experts 14.1 instead of 13.6,
// with one branch for all that is rare 14.7 (six experts x 4096 x 14336 61 instead of 56).
template <In XT> constexpr int deep() { return XT == In::F32 ? 37 : 31; }
// The weight's decode scale as m 2^e, 1 <= m < 2.
struct Decode {
    float m;
    int e;
};
__device__ __forceinline__ Decode split(float g) {
    const bool sub = g < 0x1p-126f;
    const uint32_t u = __float_as_uint(sub ? g * 0x1p64f : g);
    return Decode{__uint_as_float((u & 0x007FFFFFu) | 0x3F800000u), (int)(u >> 23) - (sub ? 191 : 127)};
}
// What brings a step's products to the result's scale is the decode scale times what undoes
// x's factor, m 2^(e - 141 + its e).  Where that exponent is outside these bounds (the
// third piece's is 22 below), and where an element is infinite or NaN, all of a row's
// elements of the step are left, for a factor in two parts (two parts for every step: 58
// us instead of 56.7 for six experts x 4096 x 14336, 21.0 instead of 20.4 for eight rows of one).
constexpr int kDownLeast = -100, kDownMost = 127;
struct Fit {
    int e;     // exponent field of the largest (at least 14); x is multiplied by 2^(141 - e)
    int left;  // elements with an exponent field below it are left; 0: none are
};

// A row's 32 elements of lane t, of those with exponent fields below `below` (kAll: of all),
// to `to`, the row's column (or the first of its three) of the step.  ge: Decode's e.
template <In XT, bool kAll>
__device__ __forceinline__ Fit put_x(const char* x, bool in, int below, int ge, uint32_t to, uint32_t col_bytes,
                                     int col, int t) {
    constexpr int kQ = XT == In::F32 ? 8 : 4;
    uint32_t w[4 * kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
        const uint4 v = in ? ld128(x + 16 * q) : make_uint4(0, 0, 0, 0);
        w[4 * q] = v.x; w[4 * q + 1] = v.y; w[4 * q + 2] = v.z; w[4 * q + 3] = v.w;
    }
    if constexpr (XT == In::F16) {
#pragma unroll
        for (int q = 0; q < 4; ++q) sts128(to + x_piece(t, col, q), w + 4 * q);
        return Fit{0, 0};
    } else {
        auto bits = [&](int i) {  // element i
            if constexpr (XT == In::F32) return w[i];
            else return i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16;
        };
        auto field = [](uint32_t u) { return (int)((u >> 23) & 255u); };
        // zeros in the place of elements with exponent fields outside lo .. hi - 1
        auto keep = [&](int lo, int hi) {
#pragma unroll
            for (int i = 0; i < 4 * kQ; ++i) {
                if constexpr (XT == In::F32) {
                    w[i] = field(w[i]) >= lo && field(w[i]) < hi ? w[i] : 0u;
                } else {
                    const int a = field(w[i] << 16), b = field(w[i]);
                    w[i] &= (a >= lo && a < hi ? 0xFFFFu : 0u) | (b >= lo && b < hi ? 0xFFFF0000u : 0u);
                }
            }
        };
        if constexpr (!kAll) keep(0, below);
        // magnitudes as whole numbers, bf16 by halves of words: the largest, and the smallest
        // but zero's less 1
        uint32_t most = 0u, least = 0xFFFFFFFFu;
#pragma unroll
        for (int i = 0; i < 4 * kQ; ++i) {
            if constexpr (XT == In::F32) {
                const uint32_t u = w[i] & 0x7FFFFFFFu;
                most = max(most, u);
                least = min(least, u - 1u);
            } else {
                const uint32_t u = w[i] & 0x7FFF7FFFu;
                most = max_halves(most, u);
                least = __viaddmin_u16x2(u, 0xFFFFFFFFu, least);
            }
        }
        if constexpr (XT != In::F32) {
            most = max(most << 16, most & 0xFFFF0000u);
            least = min(least << 16, least & 0xFFFF0000u);
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
            least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, d));
        }
        bool odd = false;  // infinities or NaN
        if constexpr (!kAll) {
            odd = __any_sync(0xFFFFFFFFu, most >= 0x7F800000u);
            if (odd) {  // the largest finite one
                most = 0u;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const uint32_t u = bits(i) & 0x7FFFFFFFu;
                    most = max(most, u < 0x7F800000u ? u : 0u);
                }
                most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
                most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
            }
        }
        const int e = max(14, (int)(most >> 23));
        Fit fit{e, 0};
        // (subnormal elements, whose last place is that of the smallest normal ones, count as
        // of field 0: within `deep` of e they are held too)
        const int small = (int)(XT == In::F32 ? (least + 1u) >> 23 : ((least >> 16) + 1u) >> 7);
        if (small < e - deep<XT>()) {
            fit.left = e - deep<XT>();
            keep(fit.left, 256);
        }
        if (kAll && most && (e == 255 || e - 141 + ge < kDownLeast || e - 141 + ge > kDownMost)) {
            fit.left = 256;
            keep(256, 256);
        }
        const float up = __uint_as_float((uint32_t)(268 - e) << 23);
        constexpr int kPieces = XT == In::F32 ? 3 : 1;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = fmul(__uint_as_float(bits(8 * q + i)), up);
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[i] = f16_pair(y[2 * i], y[2 * i + 1]);
                    if (p + 1 < kPieces) {
                        float a, b;
                        upk(f16x2_f32x2(h[i]), a, b);
                        a = (y[2 * i] - a) * 2048.0f;
                        b = (y[2 * i + 1] - b) * 2048.0f;
                        if (odd) {
                            a = fabsf(y[2 * i]) <= kFltMax ? a : 0.0f;
                            b = fabsf(y[2 * i + 1]) <= kFltMax ? b : 0.0f;
                        }
                        y[2 * i] = a;
                        y[2 * i + 1] = b;
                    }
                }
                sts128(to + p * col_bytes + x_piece(t, col + p, q), h);
            }
        }
        return fit;
    }
}
// What undoes the factor of an fp32 row's piece, column `col` of them.
template <In XT>
__device__ __forceinline__ float piece_down(int col) {
    return XT == In::F32 ? __uint_as_float((uint32_t)(127 - 11 * (col % 3)) << 23) : 1.0f;
}
// The factor of a step's products.
__device__ __forceinline__ float put_down(const Fit& fit, const Decode& g) {
    const int t = min(max(fit.e - 141 + g.e, kDownLeast), kDownMost);
    return g.m * __uint_as_float((uint32_t)(t + 127) << 23);
}
// The same of any exponent, in two parts of half of it each.  One after the other they
// neither overflow nor lose bits where the result does not (a factor at a time did: weights
// of 1e35 and x near 1, or x of 1e36 and weights of 1e-35).  Below 2^-250 nothing is left.
__device__ __forceinline__ float2 put_down2(const Fit& fit, const Decode& g) {
    const int t = max(fit.e - 141 + g.e, -250), h = t >> 1;
    return make_float2(g.m * __uint_as_float((uint32_t)(h + 127) << 23), __uint_as_float((uint32_t)(t - h + 127) << 23));
}

// This lane's 32 elements from k on of the row of x that row p takes.
template <In XT>
__device__ __forceinline__ const char* x_at(const MatvecArgs& a, int64_t p, int k) {
    return static_cast<const char*>(a.x) + ((p / a.rep) * a.K + k) * (XT == In::F32 ? 4 : 2);
}
// A lane's scales of row tile r of expert e in the first step: of row g, two bytes (of row g + 8
// 128 bytes behind, of the next step two tiles).
__device__ __forceinline__ const uint8_t* scales_at(const MatvecArgs& a, int e, int r, int g, int t) {
    return a.scales + (int64_t)e * a.scale_bytes + ((int64_t)(r >> 7) * a.kt + (t >> 1)) * lin::kSfTileBytes +
           16 * ((r & 31) + g) + 4 * ((r >> 5) & 3) + 2 * (t & 1);
}

// The products of the elements that put_x left, of a warp's steps, added to its partial
// sums: turn by turn the largest of those left decide the factor.  A function of its
// own, so that it costs the rows that leave none no registers; its codes come straight
// from memory (the ring has gone on).  x is laid out at `xs`, the factors at `down`,
// places of the warp's own.  One row x 4096 x 14336 with one such element 19.5 us instead
// of 12.4, with gelu's values of normal arguments of deviation 4 (tails to 1e-30 in most
// steps) 43, with magnitudes spread over 2^-100 .. 2^100 147.
template <In XT, int kR>
__device__ __noinline__ void add_left(const MatvecArgs& a, int e, int row0, int lo, int hi, const int* ids,
                                      int first, int ntok, Decode gd, float* part, uint32_t xs, float2* down) {
    constexpr int kPieces = XT == In::F32 ? 3 : 1, kLine = line<kR>();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    // a quad a row (those behind the last do the last one's work once more)
    const int tk = min(g, ntok - 1), col = tk * kPieces;
    const int64_t p = ids ? ids[tk] : first + tk;
    for (int step = lo + warp; step < hi; step += kWarpsMv) {
        const int k = step * kStepK + 32 * t;
        const char* x = x_at<XT>(a, p, k);
        Fit fit = put_x<XT, true>(x, k < a.K, 256, gd.e, xs + col * kXStep, kXStep, col, t);
        while (__any_sync(0xFFFFFFFFu, fit.left > 0)) {
            __syncwarp();
            fit = put_x<XT, false>(x, k < a.K, fit.left, gd.e, xs + col * kXStep, kXStep, col, t);
            if (t == 0) down[tk] = put_down2(fit, gd);
            __syncwarp();
            uint4 f[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                f[q] = g < ntok * kPieces ? lds128(xs + g * kXStep + x_piece(t, g, q)) : make_uint4(0, 0, 0, 0);
            float2 d0 = down[min(2 * t / kPieces, ntok - 1)], d1 = down[min((2 * t + 1) / kPieces, ntok - 1)];
            d0.y *= piece_down<XT>(2 * t);
            d1.y *= piece_down<XT>(2 * t + 1);
#pragma unroll 1
            for (int i = 0; i < kR; ++i) {
                uint4 w[2];
                uint32_t sc[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = row0 + 16 * i + 8 * r + g;
                    const bool in = row < a.N && k < a.K;
                    w[r] = in ? ld128(a.b + (((int64_t)e * a.N + row) * a.K + k) / 2) : make_uint4(0, 0, 0, 0);
                    sc[r] = in ? ld_u16(scales_at(a, e, row0 + 16 * i, g, t) +
                                        (int64_t)step * (2 * lin::kSfTileBytes) + 128 * r) : 0u;
                }
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_tile(sum, w[0], w[1], sc[0], sc[1], f);
                float* at = part + (2 * t) * kLine + 16 * i + g;
                at[0] = __fmaf_rn(fmul(sum[0], d0.x), d0.y, at[0]);
                at[kLine] = __fmaf_rn(fmul(sum[1], d1.x), d1.y, at[kLine]);
                at[8] = __fmaf_rn(fmul(sum[2], d0.x), d0.y, at[8]);
                at[kLine + 8] = __fmaf_rn(fmul(sum[3], d1.x), d1.y, at[kLine + 8]);
            }
        }
        __syncwarp();  // the last turn's x and factors have been read
    }
}

__device__ __forceinline__ float ld_cluster(const float* p, int rank) {
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
                 "ld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v) : "r"(smem_u32(p)), "r"(rank) : "memory");
    return v;
}

// Stores one result with its epilogue.
template <Out OT>
__device__ __forceinline__ void finish(const Epilogue& ep, float v, int64_t n_at, int64_t at) {
    if (ep.bias)
        v = fadd(v, ep.bias32 ? ld_f32(static_cast<const float*>(ep.bias) + n_at)
                              : lin::raw_value<OT>(lin::ld_raw<OT>(ep.bias, n_at)));
    float a[1] = {v};
    lin::act_apply<OT>(ep.act, a);
    if (ep.residual) a[0] = fadd(a[0], lin::raw_value<OT>(lin::ld_raw<OT>(ep.residual, at)));
    lin::store_out<OT>(ep.out, at, a[0]);
}

template <In XT, int kR>
__global__ void __launch_bounds__(32 * kWarpsMv, 2) k_matvec4(const __grid_constant__ MatvecArgs a) {
    constexpr int kRows = 16 * kR, kLine = line<kR>(), kSlot = kRows * kStepBytes, kRing = ring<kR>();
    constexpr int kTok = tokens<XT>(), kPieces = XT == In::F32 ? 3 : 1;
    extern __shared__ __align__(128) unsigned char s_ring[];
    __shared__ __align__(16) float s_sum[8 * kLine];
    __shared__ __align__(8) uint64_t s_full[kWarpsMv][kRing];
    __shared__ int s_ids[kMaxRows];
    __shared__ int s_count, s_fail, s_again;
    float* s_down = reinterpret_cast<float*>(s_ring + ring_bytes<kR>() + kXBytes + 64);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int S = a.splits, rank = (int)(blockIdx.x % S), block = (int)(blockIdx.x / S);
    const int row0 = block * kRows;
    if (lane == 0) {
        for (int b = 0; b < kRing; ++b) mma::bar_init(&s_full[warp][b], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 0) s_fail = s_again = 0;
    const uint32_t s_x = smem_u32(s_ring) + ring_bytes<kR>();
    if (tid < 16) reinterpret_cast<uint32_t*>(s_ring + ring_bytes<kR>() + kXBytes)[tid] = 0u;
    __syncthreads();
    chain_wait();
    chain_release();
    int first = blockIdx.y * kTok, count = min(kTok, a.M - first), e = 0;
    if (a.ids) {
        // the rows of this expert from blockIdx.y on, in order
        for (int q = tid; q < a.M; q += 32 * kWarpsMv) s_ids[q] = ld_s32(a.ids + q);
        __syncthreads();
        first = 0;
        e = s_ids[blockIdx.y];
        if ((unsigned)e >= (unsigned)a.G) return;  // nobody's row
        bool seen = false;
        for (int q = tid; q < (int)blockIdx.y; q += 32 * kWarpsMv) seen |= s_ids[q] == e;
        if (__syncthreads_or(seen)) return;  // the expert's first row handles it
        if (warp == 0) {
            int n = 0;
            for (int q0 = blockIdx.y; q0 < a.M; q0 += 32) {
                const bool mine = q0 + lane < a.M && s_ids[q0 + lane] == e;
                const uint32_t all = __ballot_sync(0xFFFFFFFFu, mine);
                // the list grows behind what has been read
                if (mine) s_ids[n + __popc(all & ((1u << lane) - 1u))] = q0 + lane;
                n += __popc(all);
                __syncwarp();
            }
            if (lane == 0) s_count = n;
        }
        __syncthreads();
        count = s_count;
    }
    const int nsteps = (a.K + kStepK - 1) / kStepK;
    const int lo = nsteps * rank / S, hi = nsteps * (rank + 1) / S;
    // this lane's scales: of rows g and g + 8 of row tile i, two bytes of tile t / 2 of a step
    const uint8_t* scales[kR];
#pragma unroll
    for (int i = 0; i < kR; ++i) {
        const int r = row0 + 16 * i;
        scales[i] = r < a.N ? scales_at(a, e, r, g, t) : nullptr;
    }
    // the steps in which this lane's 32 elements lie below K
    const int mine = min(hi, (a.K - 32 * t + kStepK - 1) / kStepK);
    const uint32_t lane_at = smem_u32(s_ring) + warp * kRing * kSlot + g * kStepBytes + 16 * t;
    uint32_t slot = 0, parity = 0;  // of the next step
    bool bad = false;
    const float gb = fdiv(1.0f, global_scale(ld_f32(a.ep.b_amax + e), a.ep.six_bound));
    const Decode gd = split(gb);
    // step's codes into ring slot b
    auto fetch = [&](int step, uint32_t b) {
        if (lane == 0 && step < hi) {
            mbar_expect_tx(&s_full[warp][b], kSlot);
            tma_load_2d(s_ring + (warp * kRing + b) * kSlot, &a.codes, step * kStepBytes, e * a.N + row0,
                        &s_full[warp][b]);
        }
    };
    for (int c0 = 0; c0 < count; c0 += kTok) {
        const int ntok = min(kTok, count - c0), cols = ntok * kPieces;
        float acc[kR][4];
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
        uint32_t sc[kR][2];
        auto load_scales = [&](int step) {
#pragma unroll
            for (int i = 0; i < kR; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    sc[i][r] = step < mine && scales[i] ?
                                   ld_u16(scales[i] + (int64_t)step * (2 * lin::kSfTileBytes) + 128 * r) : 0u;
        };
        {
            uint32_t b = slot;
#pragma unroll
            for (int j = 0; j < kRing; ++j) {
                fetch(lo + warp + j * kWarpsMv, b);
                b = b + 1 == kRing ? 0 : b + 1;
            }
        }
        load_scales(lo + warp);
        // x by as many steps at a time as its place in shared memory holds
        const int seg = kXBytes / kXStep / cols / kWarpsMv * kWarpsMv;
        const uint32_t col_bytes = (uint32_t)(seg * kXStep);
        for (int s0 = lo; s0 < hi; s0 += seg) {
            const int steps = min(seg, hi - s0);
            bool left = false;
            // a quad of lanes a row and step; whole warps go round together
            for (int u = warp * 8 + g; u < (ntok * steps + 7) / 8 * 8; u += kWarpsMv * 8) {
                const int tk = min(u / steps, ntok - 1), st = min(u - tk * steps, steps - 1);
                const int64_t p = a.ids ? s_ids[c0 + tk] : first + c0 + tk;
                const int k = (s0 + st) * kStepK + 32 * t;
                const Fit fit = put_x<XT, true>(x_at<XT>(a, p, k), k < a.K, 256, gd.e,
                                                s_x + tk * kPieces * col_bytes + st * kXStep, col_bytes,
                                                tk * kPieces, t);
                left |= fit.left > 0;
                if (XT != In::F16 && t == 0) s_down[tk * seg + st] = put_down(fit, gd);
            }
            if (left) s_again = 1;
            __syncthreads();
            // a column that is not there reads the step of zeros
            const bool live = g < cols;
            const float pd0 = piece_down<XT>(2 * t), pd1 = piece_down<XT>(2 * t + 1);
            const uint32_t xs = live ? s_x + g * col_bytes : s_x + kXBytes;
            for (int step = s0 + warp; step < s0 + steps; step += kWarpsMv) {
                uint32_t two[kR][2];
#pragma unroll
                for (int i = 0; i < kR; ++i)
#pragma unroll
                    for (int r = 0; r < 2; ++r) two[i][r] = sc[i][r];
                // Where they are asked for: with four row tiles here (six experts x 4096 x 14336 56.7
                // us; behind the wait 62, registers spill), else behind the wait for the codes
                // (14336 x 4096 11.3, here 11.8: the fence below waits for loads under way).
                if constexpr (kR == 4) load_scales(step + kWarpsMv);
                const uint32_t xa = live ? xs + (step - s0) * kXStep : xs;
                uint4 f[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) f[q] = lds128(xa + (live ? x_piece(t, g, q) : 16 * q));
                float d0 = 1.0f, d1 = 1.0f;  // of the two columns that this lane has products of
                if constexpr (XT != In::F16) {
                    d0 = s_down[min(2 * t / kPieces, ntok - 1) * seg + step - s0] * pd0;
                    d1 = s_down[min((2 * t + 1) / kPieces, ntok - 1) * seg + step - s0] * pd1;
                }
                if (!lin::warp_wait(&s_full[warp][slot], parity)) bad = true;  // goes on: every copy is waited for
                if constexpr (kR < 4) load_scales(step + kWarpsMv);
                const uint32_t at = lane_at + slot * kSlot;
#pragma unroll
                for (int i = 0; i < kR; ++i) {
                    const uint4 lo4 = lds128(at + 16 * i * kStepBytes), hi4 = lds128(at + (16 * i + 8) * kStepBytes);
                    float sum[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum[j] = XT == In::F16 ? acc[i][j] : 0.0f;
                    mma_tile(sum, lo4, hi4, two[i][0], two[i][1], f);
                    if constexpr (XT == In::F16) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][j] = sum[j];
                    } else {
                        acc[i][0] = __fmaf_rn(sum[0], d0, acc[i][0]);
                        acc[i][1] = __fmaf_rn(sum[1], d1, acc[i][1]);
                        acc[i][2] = __fmaf_rn(sum[2], d0, acc[i][2]);
                        acc[i][3] = __fmaf_rn(sum[3], d1, acc[i][3]);
                    }
                }
                // every lane has its codes: the slot is free (without the fence a copy issued
                // right behind the loads was seen to overtake them)
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                fetch(step + kRing * kWarpsMv, slot);
                if (++slot == kRing) {
                    slot = 0;
                    parity ^= 1u;
                }
            }
            __syncthreads();  // this part of x has been read
        }
        if (bad) s_fail = 1;
        // partial sums, column-major, over this warp's ring, whose copies have all been
        // waited for
        static_assert(kRing * kSlot >= 8 * kLine * 4, "partial sums");
        float* part = reinterpret_cast<float*>(s_ring + warp * kRing * kSlot);
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            part[(2 * t) * kLine + 16 * i + g] = acc[i][0];
            part[(2 * t + 1) * kLine + 16 * i + g] = acc[i][1];
            part[(2 * t) * kLine + 16 * i + 8 + g] = acc[i][2];
            part[(2 * t + 1) * kLine + 16 * i + 8 + g] = acc[i][3];
        }
        if constexpr (XT != In::F16) {
            if (s_again)  // put_x left elements of this chunk's rows
                add_left<XT, kR>(a, e, row0, lo, hi, a.ids ? s_ids + c0 : nullptr, first + c0, ntok, gd, part,
                                 s_x + warp * (kXBytes / kWarpsMv), reinterpret_cast<float2*>(s_down) + warp * 8);
        }
        __syncthreads();
        for (int idx = tid; idx < ntok * kRows; idx += 32 * kWarpsMv) {
            const int r = idx % kRows, tk = idx / kRows;
            float v = 0.0f;
#pragma unroll
            for (int p = XT == In::F32 ? 2 : 0; p >= 0; --p) {  // the smallest piece first
                const int at = (XT == In::F32 ? 3 * tk + p : tk) * kLine + r;
#pragma unroll
                for (int w = 0; w < kWarpsMv; ++w)
                    v = fadd(v, reinterpret_cast<const float*>(s_ring + w * kRing * kSlot)[at]);
            }
            s_sum[tk * kLine + r] = s_fail ? __int_as_float(0x7FC00000) : v;
        }
        lin::tile_sync(S);
        for (int idx = rank * 32 * kWarpsMv + tid; idx < ntok * kRows; idx += S * 32 * kWarpsMv) {
            const int r = idx % kRows, tk = idx / kRows;
            const int row = row0 + r;
            float v = s_sum[tk * kLine + r];
            if (S > 1) {
                v = 0.0f;
                for (int k = 0; k < S; ++k) v = fadd(v, ld_cluster(s_sum + tk * kLine + r, k));
            }
            if (row >= a.N) continue;
            if (XT == In::F16) v = fmul(v, gb);
            const int64_t p = a.ids ? s_ids[c0 + tk] : first + c0 + tk;
            const int64_t at = p * a.N + row, n_at = (int64_t)e * a.N + row;
            switch (static_cast<Out>(a.out_dt)) {
                case Out::BF16: finish<Out::BF16>(a.ep, v, n_at, at); break;
                case Out::F16: finish<Out::F16>(a.ep, v, n_at, at); break;
                default: finish<Out::F32>(a.ep, v, n_at, at); break;
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the ring is TMA's again
        if (tid == 0) s_again = 0;
        lin::tile_sync(S);  // the sums have been read
    }
}

}  // namespace matvec
}  // namespace fos
