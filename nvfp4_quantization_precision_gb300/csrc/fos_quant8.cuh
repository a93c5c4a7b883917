// fos_quant8.cuh -- a tensor, or the gradient of an activation, written in the
// 8-bit block format along its rows and along its columns from one read, with
// the column sums (the bias gradient).
//
//   d = x                      (quantize8)
//   d = dout * act'(pre)       (act_backward)
//   codes, scales              32-element blocks of the rows of d
//   codes_t, scales_t          32-element blocks of the rows of d^T, that is 32
//                              consecutive rows of one column; rows past the
//                              end count as zeros up to a multiple of 32
//   sums[c]                    sum of column c
//
// Bound by HBM: e (or 2e) bytes read per element, 2 + 1/16 written, e more for
// d itself.  Measured (bf16, a device copy reaches 6.78 TB/s): 14336 x 4096, both
// directions, 41.1 us, 5.8 TB/s (86 %); silu gradient with its column sums, 8192 x
// 14336, 122 us, 5.8 TB/s (86 %; relu 119, gelu_tanh 128, gelu 139 us); 1000 x
// 2048 f16 10.0 us, two launches and one tile's latency.
// A CTA takes a tile of 128 rows x 128 columns: thread t reads 16-element
// segments (t mod 8) of rows t / 8 + 32 i, so a warp reads four whole 256-byte
// row pieces; two neighbouring lanes hold one row block.  (Tiles of 64 columns,
// twice as many CTAs, whose rows are single lines, took the silu gradient 6 %
// longer.)  For the columns the tile passes through shared memory in fp32 (64 KB, three CTAs an SM); lane l then takes rows 32 (l
// mod 4) .. + 31 of column l / 4 of its warp's eight, so four lanes write the
// 128 code bytes of a column as one line and their four scale bytes as one
// word.  Element (r, c) sits in 16-byte chunk ((c / 4 ^ (c / 32) mod 4) + 2 (r /
// 32)) mod 32 of row r: the eight lanes of a store phase (one row, segments 0
// .. 7) and the 32 lanes of a load (four row groups, eight columns) then touch
// every bank once.
#pragma once

#include "fos_act.cuh"
#include "fos_block8.cuh"

namespace fos {

struct Quant8Args {
    const void* x;       // [rows, cols]: the tensor, or dout
    const void* pre;     // act_backward: the pre-activation
    void* d;             // optional: d rounded to the data's type
    uint8_t* codes;      // optional, with scales
    uint8_t* scales;
    uint8_t* codes_t;    // optional, with scales_t: [cols, rows_pad]
    uint8_t* scales_t;
    float* part;         // optional: [row tiles, cols] column sums of the row tiles
    int64_t rows, cols;
    int64_t rows_pad;    // rows rounded up to a multiple of 32
    int64_t tiles_c;
    int64_t pc4, pc4_t;  // tiled scales: 4-block tiles per tile-row
    int tiled;
    int wave;            // CTAs the device holds at once
};

constexpr int kQ8Tile = 128;  // rows and columns of a tile
constexpr int kQ8Threads = 256;
constexpr size_t kQ8Smem = kQ8Tile * kQ8Tile * sizeof(float);

// 16-byte chunk of column c in a row of row group rb.
__device__ __forceinline__ int q8_chunk(int c, int rb) {
    return (((c >> 2) ^ ((c >> 5) & 3)) + 2 * rb) & 31;
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

template <In IT, Act A>
__global__ void __launch_bounds__(kQ8Threads, 3) k_quant8(const Quant8Args a) {
    chain_wait();
    chain_release();
    extern __shared__ __align__(16) float s_tile[];
    constexpr int64_t kElt = (IT == In::F32) ? 4 : 2;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t tr = blockIdx.x / a.tiles_c, tc = blockIdx.x - tr * a.tiles_c;
    const int64_t r0 = tr * kQ8Tile, c0 = tc * kQ8Tile;
    const bool cols_wanted = a.codes_t || a.part;
    {
        const int seg = tid & 7, rl = tid >> 3;
        const bool col_in = c0 + seg * 16 < a.cols;
        // row segments in flight: what 80 registers hold
        constexpr int kAhead = (IT == In::F32) ? 1 : (A == Act::NONE ? 4 : 2);
        Raw<IT> x[kAhead], p[kAhead];
        auto load = [&](int i, Raw<IT>& xr, Raw<IT>& pr) {
            const int64_t row = r0 + rl + 32 * i;
            if (col_in && row < a.rows) {
                const int64_t at = (row * a.cols + c0 + seg * 16) * kElt;
                load_seg<IT, L2::FIRST>(xr, static_cast<const char*>(a.x) + at);
                if constexpr (A != Act::NONE)
                    load_seg<IT, L2::FIRST>(pr, static_cast<const char*>(a.pre) + at);
            } else {
                zero_seg(xr);
                if constexpr (A != Act::NONE) zero_seg(pr);
            }
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load(i, x[i], p[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = i % kAhead;
            const int64_t row = r0 + rl + 32 * i;
            const bool in = col_in && row < a.rows;
            uint64_t d[8];
            widen<IT>(x[b], d);
            if constexpr (A != Act::NONE) {
                uint64_t pv[8];
                widen<IT>(p[b], pv);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = mul2(d[j], act_slope2<A, IT == In::F32>(pv[j]));
            }
            if (i + kAhead < 4) load(i + kAhead, x[b], p[b]);
            if (a.codes) {
                float m = seg_amax(d);
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                if (in) {
                    const uint32_t sc = scale8_code(m);
                    uint32_t w[4];
                    encode8(d, scale8_inv(sc), w);
                    st128(a.codes + row * a.cols + c0 + seg * 16, w);
                    if ((seg & 1) == 0)
                        st8(a.scales + scale8_at(a.tiled, row, (c0 >> 5) + (seg >> 1),
                                                 a.cols / 32, a.pc4), sc);
                }
            }
            if (a.d && in)
                store_seg<IT>(static_cast<char*>(a.d) + (row * a.cols + c0 + seg * 16) * kElt, d);
            if (cols_wanted) {
                float* line = s_tile + (rl + 32 * i) * kQ8Tile;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float4 v;
                    upk(d[2 * k], v.x, v.y);
                    upk(d[2 * k + 1], v.z, v.w);
                    *reinterpret_cast<float4*>(line + 4 * q8_chunk(seg * 16 + 4 * k, i)) = v;
                }
            }
        }
    }
    {
        // the tile a wave from here on its way to L2, one row's half a thread:
        // its CTA then loads it at L2's latency (14336 x 4096 bf16: 44.6 -> 41.0
        // us, the silu gradient of 8192 x 14336: 133 -> 122 us)
        const int64_t nt = (int64_t)blockIdx.x + a.wave, ntr = nt / a.tiles_c, ntc = nt - ntr * a.tiles_c;
        const int64_t row = ntr * kQ8Tile + (tid >> 1);
        const int64_t c = ntc * kQ8Tile + (tid & 1) * (kQ8Tile / 2);
        if (row < a.rows && c < a.cols) {
            const int64_t at = (row * a.cols + c) * kElt;
#pragma unroll
            for (int l = 0; l < kElt / 2; ++l) {
                if (c + l * (128 / kElt) >= a.cols) break;
                prefetch_l2(static_cast<const char*>(a.x) + at + 128 * l);
                if constexpr (A != Act::NONE)
                    prefetch_l2(static_cast<const char*>(a.pre) + at + 128 * l);
            }
        }
    }
    if (a.tiled) {
        const uint32_t t = blockIdx.x * kQ8Threads + tid, n = gridDim.x * kQ8Threads;
        if (a.codes) clear_tiled_pad(a.scales, a.rows, a.cols / 32, a.pc4, t, n);
        if (a.codes_t) clear_tiled_pad(a.scales_t, a.cols, a.rows_pad / 32, a.pc4_t, t, n);
    }
    if (!cols_wanted) return;
    __syncthreads();
    const int rb = lane & 3;
    const int64_t rblk = r0 + 32 * rb;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int cl = half * 64 + warp * 8 + (lane >> 2);
        const int64_t c = c0 + cl;
        const float* col = s_tile + 32 * rb * kQ8Tile + 4 * q8_chunk(cl, rb) + (cl & 3);
        uint64_t v[2][8];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i >> 3][i & 7] = pk(col[(2 * i) * kQ8Tile], col[(2 * i + 1) * kQ8Tile]);
        if (a.codes_t && c < a.cols && rblk < a.rows_pad) {
            const uint32_t sc = scale8_code(fmaxf(seg_amax(v[0]), seg_amax(v[1])));
            const float inv = scale8_inv(sc);
            uint32_t w[2][4];
            encode8(v[0], inv, w[0]);
            encode8(v[1], inv, w[1]);
            const uint32_t o[8] = {w[0][0], w[0][1], w[0][2], w[0][3],
                                   w[1][0], w[1][1], w[1][2], w[1][3]};
            st256(a.codes_t + c * a.rows_pad + rblk, o);
            st8(a.scales_t + scale8_at(a.tiled, c, rblk >> 5, a.rows_pad / 32, a.pc4_t), sc);
        }
        if (a.part) {
            uint64_t s2 = add2(v[0][0], v[1][0]);
#pragma unroll
            for (int j = 1; j < 8; ++j) s2 = add2(s2, add2(v[0][j], v[1][j]));
            float s, t;
            upk(s2, s, t);
            s = fadd(s, t);
            s = fadd(s, __shfl_xor_sync(0xFFFFFFFFu, s, 1));
            s = fadd(s, __shfl_xor_sync(0xFFFFFFFFu, s, 2));
            if (rb == 0 && c < a.cols) a.part[tr * a.cols + c] = s;
        }
    }
}

}  // namespace fos
