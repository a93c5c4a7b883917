// fos_norm.cuh -- root-mean-square norm with the residual's addition and an
// 8-bit block-scaled output, and its backward pass.
//
//   forward   h = x + residual; rstd = 1 / sqrt(mean(h^2) + eps);
//             y = h * rstd * w; codes and scales of y's rows (fos_block8.cuh)
//   backward  g = dy * w; xh = h * rstd; dx = rstd * (g - h * (rstd * mean(g * xh))) + dh;
//             dw[c] = sum over rows of dy * xh
//
// Both are bound by HBM: forward e bytes read per element of e bytes (2 e with
// the residual) and 1 + 1/32 written (e more for h), backward 2e or 3e read and
// e written.  So a row is read once and lives in registers: a group of kT
// threads owns a row, thread t the 16-element segments t, t + kT, ..., the row's
// sum crosses the group by shuffles and one barrier, and the next row's loads are
// issued before the current row is finished.  Two neighbouring lanes hold one
// 32-element block.  A thread holds one or two segments (one in the backward
// pass, whose weight gradient takes 16 more registers a segment); rows of up to
// 1024 elements go one to a warp, without a barrier.
//
// Measured, against a device copy's 6.78 TB/s (bf16 unless named):
//   forward   16384 x 7168 with residual, h, codes, scales: 127.5 us, 6.47 TB/s
//             (95 %); 8192 x 4096 without residual and h: 19.0 us
//   backward  8192 x 4096 with dh and dw: 45.0 us, 5.97 TB/s (88 %);
//             1021 x 7168 fp32 without dh: 18.8 us, 4.69 TB/s (69 %; 6.7 rows a
//             CTA, then 2.5 us for the sum of the weight gradient's partial rows)
//   one row of 4096: 2.1 us, the chain of a launch, two reads of memory and a
//             barrier
// The variant goes by the row's width alone, so that a row's result does not
// depend on how many others are with it.

#pragma once

#include "fos_block8.cuh"
#include "fos_kernels.cuh"

namespace fos {

struct NormArgs {
    const void* x;
    const void* res;    // optional
    const void* w;
    void* h;            // optional: x + res rounded to the data's type
    void* y;            // optional: the norm's output rounded to the data's type
    uint8_t* codes;     // optional, with scales
    uint8_t* scales;
    float* rstd;        // optional, [rows]
    int64_t rows;
    int64_t cols;
    int64_t pc4;        // tiled scales: 4-block tiles per tile-row
    float inv_cols;     // 1 / cols, rounded, and
    float inv_cols_lo;  // what the rounding leaves out
    float eps;
    int w32;            // weight is fp32 (else the data's type)
    int tiled;
};

// Sum over groups of kLanes lanes (a fixed tree; every lane gets it).
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int m = kLanes / 2; m >= 1; m >>= 1) v = fadd(v, __shfl_xor_sync(0xFFFFFFFFu, v, m));
    return v;
}
// The sum of kW warps' sums in shared memory, in every lane.
template <int kW>
__device__ __forceinline__ float parts_sum(const float* part) {
    return lanes_sum<kW>(part[threadIdx.x & (kW - 1)]);
}

// s / cols + add.  1 / cols rounded to fp32 is off by the same 2^-25 or less in every
// row (7168: 4.5e-8, half of it in rstd, as much as all roundings of the row together),
// which one more multiply-add takes out (of a finite sum: an infinite one stays that).
__device__ __forceinline__ float row_mean(float s, float inv, float inv_lo, float add) {
    return __fmaf_rn(s, inv, __fmaf_rn(fmaxf(fminf(s, kFltMax), -kFltMax), inv_lo, add));
}

// 1 / sqrt(m): the hardware's approximation (2 ulp) and one Newton step, whose
// residual 1 - m r^2 carries the rounding of m r along (a row's rstd: 3.6e-8 root
// mean square instead of 3.9e-8, at no measurable time).
__device__ __forceinline__ float rsqrt1(float m) {
    const float r = rsqrtf(m);
    const float t = fmul(m, r);
    const float e = __fmaf_rn(-__fmaf_rn(m, r, -t), r, __fmaf_rn(-t, r, 1.0f));
    // a zero or infinite mean has no finite correction
    return isfinite(e) ? __fmaf_rn(fmul(0.5f, r), e, r) : r;
}

// Sum of the squares of 16 values, added to two packed accumulators.
__device__ __forceinline__ void add_squares(const uint64_t (&v)[8], uint64_t& a0, uint64_t& a1) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        a0 = fma2(v[j], v[j], a0);
        a1 = fma2(v[j + 1], v[j + 1], a1);
    }
}

// y = (h * w) * rstd.  In this order the first product of 16-bit h and w is exact
// in 32 bits, so that y carries rstd's error and one rounding of its own; h * rstd
// first would round twice.  h * w leaves the range of 32 bits only where the row's
// sum of squares already has, or with weights beyond 10^19.  Of 705 M codes (8192 x
// 7168 with a residual) 437 differ from the exact ones, 462 of a plain fp32 form.
// (Carrying the rounding errors of the sum, the mean, rstd and the products along: 343,
// at 16384 x 7168 129.4 instead of 127.7 us, 8192 x 4096 40.2 instead of 38.9.)
__device__ __forceinline__ void normed(const uint64_t (&h)[8], const uint64_t (&w)[8], float r,
                                       uint64_t (&y)[8]) {
    const uint64_t r2 = pk(r, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = mul2(mul2(h[j], w[j]), r2);
}

// Outputs of one segment of a finished row; every lane of a pair takes part.
template <In IT>
__device__ __forceinline__ void emit_norm(const NormArgs& a, int64_t row, int64_t seg, bool in,
                                          const uint64_t (&h)[8], const uint64_t (&w)[8],
                                          float r) {
    constexpr int64_t kElt = (IT == In::F32) ? 4 : 2;
    uint64_t y[8];
    normed(h, w, r, y);
    float m = seg_amax(y);
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    if (!in) return;
    const int64_t at = row * a.cols + seg * 16;
    if (a.h) store_seg<IT>(static_cast<char*>(a.h) + at * kElt, h);
    if (a.y) store_seg<IT>(static_cast<char*>(a.y) + at * kElt, y);
    if (a.codes) {
        const uint32_t sc = scale8_code(m);
        uint32_t c[4];
        encode8(y, scale8_inv(sc), c);
        st128(a.codes + at, c);
        if ((seg & 1) == 0)
            st8(a.scales + scale8_at(a.tiled, row, seg >> 1, a.cols / 32, a.pc4), sc);
    }
}

// `bytes` from p on (both multiples of 16) on their way to L2.
__device__ __forceinline__ void fetch_l2(const void* p, int64_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"((uint32_t)bytes)
                 : "memory");
}

template <In IT, bool RES>
__device__ __forceinline__ void load_row_seg(const NormArgs& a, int64_t row, int64_t seg, bool in,
                                             Raw<IT>& x, Raw<IT>& r) {
    constexpr int64_t kElt = (IT == In::F32) ? 4 : 2;
    const int64_t at = (row * a.cols + seg * 16) * kElt;
    if (in) {
        load_seg<IT, L2::FIRST>(x, static_cast<const char*>(a.x) + at);
        if constexpr (RES) load_seg<IT, L2::FIRST>(r, static_cast<const char*>(a.res) + at);
    } else {
        zero_seg(x);
        if constexpr (RES) zero_seg(r);
    }
}

template <In IT, bool RES>
__device__ __forceinline__ void row_values(const Raw<IT>& x, const Raw<IT>& r, uint64_t (&h)[8]) {
    widen<IT>(x, h);
    if constexpr (RES) {
        uint64_t b[8];
        widen<IT>(r, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = add2(h[j], b[j]);
    }
}

// A row per warp (kT = 32) or per group of 64 .. 512 threads, CTAs of at least 256
// threads.  Without a residual a row is small against the memory's latency (what
// the next row's loads keep in flight is 24 KB an SM, and 5.3 TB/s with 800 ns take
// 28), so the row after it is fetched to L2 as well (33.5 M elements without / with:
// bf16, 2048 wide 25.8 / 22.4 us, 4096 21.5 / 19.4, 16384 21.9 / 20.3; fp32, 2048
// wide 31.7 / 28.7, where rows of 4096 and more lose 0.4 to 1.3 us by it, as a
// residual does: bf16 16384 x 7168 127 / 136).
template <In IT, bool RES, int kT, int kSeg>
__global__ void __launch_bounds__(kT < 256 ? 256 : kT) k_rms_norm(const NormArgs a) {
    chain_wait();
    chain_release();
    constexpr int kCta = kT < 256 ? 256 : kT;      // threads of a CTA
    constexpr int kGroups = kCta / kT;             // rows of a CTA at a time
    constexpr int kW = kT / 32;                    // warps of a row
    constexpr bool kFar = !RES && (IT != In::F32 || kT < 256);
    __shared__ float s_part[2][kCta / 32];
    const int t = threadIdx.x % kT, g = threadIdx.x / kT;
    const int64_t nseg = a.cols / 16;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    uint64_t w[kSeg][8];
    bool in[kSeg];
    Raw<IT> x[kSeg], r[kSeg];
    int64_t row = (int64_t)blockIdx.x * kGroups + g;
#pragma unroll
    for (int k = 0; k < kSeg; ++k) {
        in[k] = t + k * kT < nseg;
        load_row_seg<IT, RES>(a, row, t + k * kT, in[k] && row < a.rows, x[k], r[k]);
    }
#pragma unroll
    for (int k = 0; k < kSeg; ++k) {
        if (in[k]) load_weight<IT>(a.w, (t + k * kT) * 16, a.w32, w[k]);
        else
#pragma unroll
            for (int j = 0; j < 8; ++j) w[k][j] = 0;
    }
    if (a.tiled && a.codes)
        clear_tiled_pad(a.scales, a.rows, a.cols / 32, a.pc4, blockIdx.x * kCta + threadIdx.x,
                        gridDim.x * kCta);
    // all groups of a CTA make the same number of turns (they share barriers)
    const int64_t first = (int64_t)blockIdx.x * kGroups;
    int parity = 0;
    for (int64_t base = first; base < a.rows; base += step, row += step, parity ^= 1) {
        uint64_t h[kSeg][8], a0 = 0, a1 = 0;
#pragma unroll
        for (int k = 0; k < kSeg; ++k) {
            row_values<IT, RES>(x[k], r[k], h[k]);
            add_squares(h[k], a0, a1);
            load_row_seg<IT, RES>(a, row + step, t + k * kT, in[k] && row + step < a.rows, x[k],
                                  r[k]);
        }
        if constexpr (kFar) {
            constexpr int kElt = (IT == In::F32) ? 4 : 2;
            const int64_t far = row + 2 * step;
            if (t == 0 && far < a.rows)
                fetch_l2(static_cast<const char*>(a.x) + far * a.cols * kElt, a.cols * kElt);
        }
        float p0, p1, p2, p3;
        upk(a0, p0, p1);
        upk(a1, p2, p3);
        float s = lanes_sum<32>(fadd(fadd(p0, p1), fadd(p2, p3)));
        if constexpr (kW > 1) {
            const int wid = threadIdx.x >> 5;
            if ((threadIdx.x & 31) == 0) s_part[parity][wid] = s;
            __syncthreads();
            s = parts_sum<kW>(s_part[parity] + g * kW);
        }
        const float rs = rsqrt1(row_mean(s, a.inv_cols, a.inv_cols_lo, a.eps));
        if (t == 0 && a.rstd && row < a.rows) a.rstd[row] = rs;
#pragma unroll
        for (int k = 0; k < kSeg; ++k)
            emit_norm<IT>(a, row, t + k * kT, in[k] && row < a.rows, h[k], w[k], rs);
    }
}

// Rows of more than 16384 elements, which no longer fit a CTA's registers: a CTA
// per row reads it twice, the second time from L2 (a row of x and residual is at
// most a few MB).
template <In IT, bool RES>
__global__ void __launch_bounds__(512) k_rms_norm_wide(const NormArgs a) {
    chain_wait();
    chain_release();
    constexpr int kT = 512;
    __shared__ float s_part[2][kT / 32];
    const int t = threadIdx.x;
    const int64_t nseg = a.cols / 16;
    if (a.tiled && a.codes)
        clear_tiled_pad(a.scales, a.rows, a.cols / 32, a.pc4, blockIdx.x * kT + t,
                        gridDim.x * kT);
    int parity = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
        uint64_t a0 = 0, a1 = 0;
        for (int64_t sg = t; sg < nseg; sg += kT) {
            Raw<IT> x, r;
            uint64_t h[8];
            load_row_seg<IT, RES>(a, row, sg, true, x, r);
            row_values<IT, RES>(x, r, h);
            add_squares(h, a0, a1);
        }
        float p0, p1, p2, p3;
        upk(a0, p0, p1);
        upk(a1, p2, p3);
        float s = lanes_sum<32>(fadd(fadd(p0, p1), fadd(p2, p3)));
        if ((t & 31) == 0) s_part[parity][t >> 5] = s;
        __syncthreads();
        s = parts_sum<kT / 32>(s_part[parity]);
        const float rs = rsqrt1(row_mean(s, a.inv_cols, a.inv_cols_lo, a.eps));
        if (t == 0 && a.rstd) a.rstd[row] = rs;
        for (int64_t base = 0; base < nseg; base += kT) {  // whole warps for the block shuffles
            const int64_t sg = base + t;
            const bool in = sg < nseg;
            Raw<IT> x, r;
            uint64_t h[8], w[8];
            load_row_seg<IT, RES>(a, row, sg, in, x, r);
            row_values<IT, RES>(x, r, h);
            if (in) load_weight<IT>(a.w, sg * 16, a.w32, w);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 0;
            emit_norm<IT>(a, row, sg, in, h, w, rs);
        }
    }
}

// ------------------------------------------------------------------ backward
struct NormBwdArgs {
    const void* dy;
    const void* h;
    const void* dh;       // optional
    const float* rstd;
    const void* w;
    void* dx;
    float* part;          // [gridDim.x, cols] partial weight gradients, or null
    int64_t rows, cols;
    float inv_cols;       // as in NormArgs
    float inv_cols_lo;
    int w32;
};

template <In IT, bool DH>
__device__ __forceinline__ void load_bwd_seg(const NormBwdArgs& a, int64_t at, bool in, Raw<IT>& dy,
                                             Raw<IT>& h, Raw<IT>& dh) {
    constexpr int64_t kElt = (IT == In::F32) ? 4 : 2;
    if (in) {
        load_seg<IT, L2::FIRST>(dy, static_cast<const char*>(a.dy) + at * kElt);
        load_seg<IT, L2::FIRST>(h, static_cast<const char*>(a.h) + at * kElt);
        if constexpr (DH) load_seg<IT, L2::FIRST>(dh, static_cast<const char*>(a.dh) + at * kElt);
    } else {
        zero_seg(dy);
        zero_seg(h);
        if constexpr (DH) zero_seg(dh);
    }
}

// dx of one segment from g = dy * w and c = rstd mean(g xh): (g - h c) rstd, plus dh.
// In this order every step is of g's or of dx's size, also where rows are so small
// (1e-20, with eps = 0) that rstd^3 leaves fp32's range.
template <bool DH>
__device__ __forceinline__ void bwd_dx(const uint64_t (&g)[8], const uint64_t (&h)[8],
                                       const uint64_t (&dh)[8], float rstd, float c,
                                       uint64_t (&dx)[8]) {
    const uint64_t r2 = pk(rstd, rstd), c2 = pk(-c, -c);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint64_t t = fma2(h[j], c2, g[j]);
        if constexpr (DH) dx[j] = fma2(t, r2, dh[j]);
        else dx[j] = mul2(t, r2);
    }
}

// A row per group of kT threads, one 16-element segment a thread; a CTA of 512
// threads holds 512 / kT groups.  The weight gradient of the thread's columns
// is kept in registers over all of its rows and leaves as one partial row per
// CTA (its groups are added in order through shared memory), so the sum has one
// fixed order and the second kernel one partial row per SM to add (CTAs of one
// group, four an SM with a partial row each: 46.8 instead of 45.0 us for 8192 x
// 4096).  512 threads because dw and a row in flight next to the row in work take
// 128 registers a thread.  Where one group takes the whole CTA, an SM has one row in
// work and one in flight, and the row after that is fetched to L2 (4681 x 7168
// without / with: bf16 52.8 / 38.4 us, with dh 47.4 / 45.0; fp32 with dh 92.6 /
// 84.7; narrower rows, of which an SM has more, lose by it: 8192 x 4096 45.2 /
// 46.6).
constexpr int kBwdThreads = 512;
template <In IT, int kT, bool DH>
__global__ void __launch_bounds__(kBwdThreads, 1) k_rms_bwd(const NormBwdArgs a) {
    chain_wait();
    chain_release();
    constexpr int kGroups = kBwdThreads / kT, kW = kT / 32;
    constexpr bool kFar = kGroups == 1;
    constexpr bool kAhead = IT != In::F32 || !DH;  // the next row fits the registers
    __shared__ float s_part[2][kBwdThreads / 32];
    __shared__ float s_dw[kGroups > 1 ? kBwdThreads * 16 : 1];
    const int t = threadIdx.x % kT, g = threadIdx.x / kT;
    const bool col_in = (int64_t)t * 16 < a.cols;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    uint64_t w[8], dw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = dw[j] = 0;
    int64_t row = (int64_t)blockIdx.x * kGroups + g;
    Raw<IT> dy, h, dh;
    if constexpr (kAhead)
        load_bwd_seg<IT, DH>(a, row * a.cols + t * 16, col_in && row < a.rows, dy, h, dh);
    float rstd_next = kAhead && row < a.rows ? ld_f32(a.rstd + row) : 0.0f;
    if (col_in) load_weight<IT>(a.w, (int64_t)t * 16, a.w32, w);
    int parity = 0;
    // a group runs its own rows; only its warps meet at a barrier
    for (; row < a.rows; row += step, parity ^= 1) {
        if constexpr (!kAhead) load_bwd_seg<IT, DH>(a, row * a.cols + t * 16, col_in, dy, h, dh);
        const float rstd = kAhead ? rstd_next : ld_f32(a.rstd + row);
        uint64_t v[8], hv[8], acc = 0;
        widen<IT>(dy, v);
        widen<IT>(h, hv);
        const uint64_t r2 = pk(rstd, rstd);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint64_t xh = mul2(hv[j], r2);
            dw[j] = fma2(v[j], xh, dw[j]);
            v[j] = mul2(v[j], w[j]);
            acc = fma2(v[j], xh, acc);
        }
        uint64_t dhv[8];
        if constexpr (DH) widen<IT>(dh, dhv);
        if constexpr (kAhead) {
            load_bwd_seg<IT, DH>(a, (row + step) * a.cols + t * 16, col_in && row + step < a.rows, dy,
                                 h, dh);
            if (row + step < a.rows) rstd_next = ld_f32(a.rstd + row + step);
        }
        if constexpr (kFar) {
            constexpr int kElt = (IT == In::F32) ? 4 : 2;
            const int64_t far = row + 2 * step;
            if (t < (DH ? 3 : 2) && far < a.rows) {
                const void* p = t == 0 ? a.dy : (t == 1 ? a.h : a.dh);
                fetch_l2(static_cast<const char*>(p) + far * a.cols * kElt, a.cols * kElt);
            }
        }
        float p0, p1;
        upk(acc, p0, p1);
        float s = lanes_sum<32>(fadd(p0, p1));
        if constexpr (kW > 1) {
            if ((threadIdx.x & 31) == 0) s_part[parity][threadIdx.x >> 5] = s;
            asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "n"(kT) : "memory");
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < kW; ++i) s = fadd(s, s_part[parity][g * kW + i]);
        }
        if (col_in) {
            constexpr int64_t kElt = (IT == In::F32) ? 4 : 2;
            const float c = fmul(row_mean(s, a.inv_cols, a.inv_cols_lo, 0.0f), rstd);
            uint64_t dx[8];
            bwd_dx<DH>(v, hv, dhv, rstd, c, dx);
            store_seg<IT>(static_cast<char*>(a.dx) + (row * a.cols + t * 16) * kElt, dx);
        }
    }
    if (!a.part) return;
    if constexpr (kGroups > 1) {
        float* mine = s_dw + threadIdx.x * 16;
#pragma unroll
        for (int j = 0; j < 8; ++j) upk(dw[j], mine[2 * j], mine[2 * j + 1]);
        __syncthreads();
        // column i of the CTA's partial: the groups in order
        for (int64_t i = threadIdx.x; i < a.cols; i += kBwdThreads) {
            float s = s_dw[i];
#pragma unroll
            for (int k = 1; k < kGroups; ++k) s = fadd(s, s_dw[k * kT * 16 + i]);
            a.part[(int64_t)blockIdx.x * a.cols + i] = s;
        }
    } else if (col_in) {
        store_seg<In::F32>(a.part + (int64_t)blockIdx.x * a.cols + (int64_t)t * 16, dw);
    }
}

// Rows too wide for a segment per thread: a CTA per row, two sweeps of it for
// dx (the second from L2), no weight gradient.
template <In IT>
__global__ void __launch_bounds__(512) k_rms_bwd_wide(const NormBwdArgs a) {
    chain_wait();
    chain_release();
    constexpr int kT = 512;
    constexpr int64_t kElt = (IT == In::F32) ? 4 : 2;
    __shared__ float s_part[2][kT / 32];
    const int t = threadIdx.x;
    const int64_t nseg = a.cols / 16;
    int parity = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
        const float rstd = ld_f32(a.rstd + row);
        const uint64_t r2 = pk(rstd, rstd);
        uint64_t acc = 0;
        for (int64_t sg = t; sg < nseg; sg += kT) {
            Raw<IT> dy, h;
            uint64_t v[8], hv[8], w[8];
            const int64_t at = (row * a.cols + sg * 16) * kElt;
            load_seg<IT>(dy, static_cast<const char*>(a.dy) + at);
            load_seg<IT>(h, static_cast<const char*>(a.h) + at);
            load_weight<IT>(a.w, sg * 16, a.w32, w);
            widen<IT>(dy, v);
            widen<IT>(h, hv);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc = fma2(mul2(v[j], w[j]), mul2(hv[j], r2), acc);
        }
        float p0, p1;
        upk(acc, p0, p1);
        float s = lanes_sum<32>(fadd(p0, p1));
        if ((t & 31) == 0) s_part[parity][t >> 5] = s;
        __syncthreads();
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < kT / 32; ++i) s = fadd(s, s_part[parity][i]);
        const float c = fmul(row_mean(s, a.inv_cols, a.inv_cols_lo, 0.0f), rstd);
        for (int64_t sg = t; sg < nseg; sg += kT) {
            Raw<IT> dy, h, dh;
            uint64_t v[8], hv[8], dhv[8], w[8], dx[8];
            if (a.dh) load_bwd_seg<IT, true>(a, row * a.cols + sg * 16, true, dy, h, dh);
            else {
                load_bwd_seg<IT, false>(a, row * a.cols + sg * 16, true, dy, h, dh);
                zero_seg(dh);
            }
            load_weight<IT>(a.w, sg * 16, a.w32, w);
            widen<IT>(dy, v);
            widen<IT>(h, hv);
            widen<IT>(dh, dhv);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = mul2(v[j], w[j]);
            bwd_dx<true>(v, hv, dhv, rstd, c, dx);
            store_seg<IT>(static_cast<char*>(a.dx) + (row * a.cols + sg * 16) * kElt, dx);
        }
    }
}

// Weight gradient of wide rows: CTA (strip, y) sums rows y, y + gridDim.y, ...
// of a strip of 4096 columns into partial row y.
template <In IT>
__global__ void __launch_bounds__(256) k_rms_dw_wide(const NormBwdArgs a) {
    chain_wait();
    chain_release();
    constexpr int64_t kElt = (IT == In::F32) ? 4 : 2;
    const int64_t c0 = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 16;
    if (c0 >= a.cols) return;
    uint64_t dw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = 0;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float rstd = ld_f32(a.rstd + row);
        const uint64_t r2 = pk(rstd, rstd);
        Raw<IT> dy, h;
        uint64_t v[8], hv[8];
        const int64_t at = (row * a.cols + c0) * kElt;
        load_seg<IT>(dy, static_cast<const char*>(a.dy) + at);
        load_seg<IT>(h, static_cast<const char*>(a.h) + at);
        widen<IT>(dy, v);
        widen<IT>(h, hv);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[j] = fma2(v[j], mul2(hv[j], r2), dw[j]);
    }
    store_seg<In::F32>(a.part + (int64_t)blockIdx.y * a.cols + c0, dw);
}

// ------------------------------------------------------------------ column sums
// out[c] = sum over the `parts` partial rows, in a fixed order: a CTA takes 32
// columns, its 32 warps every 32nd row each (eight of them in flight), and the
// warps' sums are added by one tree.  Bound by latency: 152 rows of 7168 (4.4 MB,
// in L2) take about 2.5 us, started ahead of the kernel before's end.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) k_column_sums(const float* part, int64_t parts,
                                                                int64_t cols, float* out);

}  // namespace fos
