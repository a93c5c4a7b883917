// fos_matvec.cuh -- few rows of 16 or 32 bits times NVFP4 weights:
//
//   out[p][n] = act(g[e] sum_k x[p / rep][k] w[e][n][k] + bias[e][n]) + residual[p][n]
//
// e = ids[p] (0 without ids), w = e2m1(code) * e4m3(scale of its 16 elements) and
// g[e] the weight's global decode scale.  x keeps its type: no rounding before the
// sum.  Bound by the weights' bytes (9/16 byte an element), close behind by the
// instructions that unpack them.
//
// A weight w is exact in bf16 and in fp16 (two significant bits times four, 2^-10
// to 2688), so the sums are formed by mma.m16n8k16 with weights as the 16 rows,
// rows of x as the 8 columns and fp32 accumulators: one instruction for 2048
// products, whose cost in the tensor cores does not show beside the unpacking.
// tcgen05 would take its operands through shared or tensor memory, two more moves
// of every unpacked weight, for tiles of 128 rows that eight columns never fill.
//   unpack   the magnitude bits eem of a code, moved to the exponent's low bits and
//            the mantissa's top bit, are 2^-126 (bf16) or 2^-14 (fp16) times its
//            value, subnormal for 0.5; nibbles i and i + 4 of a word make a pair by
//            one shift each for sign and magnitude.  An E4M3 byte moved likewise is
//            2^-120 or 2^-8 times its value.  The scale is brought to 2^119 (2^7),
//            so that code times scale is 2^-7 w, a normal bf16 (an fp16 multiple of
//            2^-17), exactly.
//   order    a lane takes 32 elements of a row (16 bytes) and gives them to eight
//            MMAs, four a time: any order of k serves as long as x has the same.
//   x fp32   is split into three bf16 of 8 significant bits each (exactly: by
//            truncation), which take three columns; two rows at a time.
// A CTA takes 64 weight rows: rows 32 i + 16 h + 0 .. 15, i = 0 .. 3, of one
// 128-row tile of scales, so that a lane's 16 bytes of scales serve four of its
// rows.  Its eight warps split K by steps of 128, and with few CTAs the CTAs of a
// cluster do too; partial sums are added in one fixed order, warps first.
// With ids, grid row p handles the rows of expert ids[p] at once if p is the first
// of them (the weights are read once), else nothing.
#pragma once

#include "fos_groups.cuh"
#include "fos_linear.cuh"

namespace fos {

struct MatvecArgs {
    const void* x;          // [M / rep, K]
    const int32_t* ids;     // [M] or null
    const uint8_t* codes;   // [G, N, K / 2]
    const uint8_t* scales;  // [G] x tiled
    Epilogue ep;            // b_amax [G]
    int64_t scale_bytes;    // of one expert
    int M, N, K, G, rep;
    int kt;                 // scale tiles along K (64 elements)
    int splits;
    int out_dt;             // Out
};

namespace matvec {

constexpr int kWarpsMv = 8, kRows = 64, kStepK = 128, kMaxRows = 1024;
constexpr int kLine = 68;  // floats of a column of partial sums: its stores touch every bank once

template <In XT> constexpr int tokens() { return XT == In::F32 ? 2 : 8; }

__device__ __forceinline__ uint4 ld128(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <In XT>
__device__ __forceinline__ uint32_t mul_pair(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (XT == In::F16) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Pairs (element i, element i + 4) of a word of eight codes, times the scale pair.
template <In XT>
__device__ __forceinline__ void unpack(uint32_t w, uint32_t s, uint32_t (&v)[4]) {
    constexpr uint32_t kSign = 0x80008000u, kMag = XT == In::F16 ? 0x0E000E00u : 0x01C001C0u;
    if constexpr (XT == In::F16) {
        v[0] = ((w << 9) & kMag) | ((w << 12) & kSign);
        v[1] = ((w << 5) & kMag) | ((w << 8) & kSign);
        v[2] = ((w << 1) & kMag) | ((w << 4) & kSign);
        v[3] = ((w >> 3) & kMag) | (w & kSign);
    } else {
        v[0] = ((w << 6) & kMag) | ((w << 12) & kSign);
        v[1] = ((w << 2) & kMag) | ((w << 8) & kSign);
        v[2] = ((w >> 2) & kMag) | ((w << 4) & kSign);
        v[3] = ((w >> 6) & kMag) | (w & kSign);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul_pair<XT>(v[i], s);
}
// Scale byte (0x00 .. 0x7E) as a pair, 2^119 (fp16 2^7) times its value.
template <In XT>
__device__ __forceinline__ uint32_t scale_pair(uint32_t byte) {
    if constexpr (XT == In::F16) {
        return mul_pair<XT>((byte & 0x7Fu) * 0x00800080u, 0x78007800u);  // 2^15
    } else {
        const uint32_t a = mul_pair<XT>((byte & 0x7Fu) * 0x00100010u, 0x7F007F00u);  // 2^127
        return mul_pair<XT>(a, 0x77807780u);                                          // 2^112
    }
}
template <In XT>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (XT == In::F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Piece `p` (0 .. 2) of an fp32 as the top half of a word: x = the sum of its pieces,
// each a truncation to 8 significant bits of what is left.  An infinity is its first
// piece, the others 0; a NaN keeps a NaN.
__device__ __forceinline__ uint32_t piece(float x, int p) {
    const float hi = __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
    if (!(fabsf(x) <= kFltMax))
        return p > 0 ? 0u : (x != x ? 0x7FC00000u : __float_as_uint(x));
    const float r = x - hi;
    const float mid = __uint_as_float(__float_as_uint(r) & 0xFFFF0000u);
    return __float_as_uint(p == 0 ? hi : p == 1 ? mid : r - mid) & 0xFFFF0000u;
}

// x's 32 elements of a lane as the MMAs' second operand, in the order of unpack().
template <In XT>
struct Frag {
    uint32_t b[4][4];  // word of codes, pair
};
template <In XT>
__device__ __forceinline__ void load_x(Frag<XT>& f, const void* x, int64_t at, int col) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (XT == In::F32) {
            const uint4 lo = ld128(static_cast<const float*>(x) + at + 8 * q);
            const uint4 hi = ld128(static_cast<const float*>(x) + at + 8 * q + 4);
            const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, h[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f.b[q][i] = (piece(__uint_as_float(l[i]), col % 3) >> 16) |
                            piece(__uint_as_float(h[i]), col % 3);
        } else {
            const uint4 w = ld128(static_cast<const unsigned short*>(x) + at + 8 * q);
            f.b[q][0] = __byte_perm(w.x, w.z, 0x5410);
            f.b[q][1] = __byte_perm(w.x, w.z, 0x7632);
            f.b[q][2] = __byte_perm(w.y, w.w, 0x5410);
            f.b[q][3] = __byte_perm(w.y, w.w, 0x7632);
        }
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
        v = fadd(v, ep.bias32 ? static_cast<const float*>(ep.bias)[n_at]
                              : lin::load_out<OT>(ep.bias, n_at));
    float a[1] = {v};
    lin::act_apply<OT>(ep.act, a);
    if (ep.residual) a[0] = fadd(a[0], lin::load_out<OT>(ep.residual, at));
    lin::store_out<OT>(ep.out, at, a[0]);
}

template <In XT>
__global__ void __launch_bounds__(32 * kWarpsMv, 2) k_matvec4(const __grid_constant__ MatvecArgs a) {
    __shared__ float s_part[kWarpsMv][8 * kLine];
    __shared__ __align__(16) float s_sum[8 * kLine];
    __shared__ int s_ids[kMaxRows];
    __shared__ int s_count;
    constexpr int kTok = tokens<XT>();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int S = a.splits, rank = (int)(blockIdx.x % S), block = (int)(blockIdx.x / S);
    const int row0 = (block >> 1) * 128 + (block & 1) * 16;  // of i = 0
    chain_wait();
    chain_release();
    if (row0 >= a.N) return;  // the second half of a last tile
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
    const uint8_t* codes = a.codes + (int64_t)e * a.N * (a.K / 2);
    const uint8_t* scales = a.scales + (int64_t)e * a.scale_bytes +
                            (int64_t)(row0 >> 7) * a.kt * lin::kSfTileBytes +
                            16 * ((row0 & 31) + g);
    // with the 2^7 that unpacked weights lack (exact, and in range: g <= FLT_MAX / 1536)
    const float gb = fmul(fdiv(1.0f, global_scale(a.ep.b_amax[e], a.ep.six_bound)), 128.0f);
    for (int c0 = 0; c0 < count; c0 += kTok) {
        const int ntok = min(kTok, count - c0);
        // this lane's column of the second operand: a row of x, or nothing
        const int tok = XT == In::F32 ? g / 3 : g;
        const bool live = tok < ntok;
        int64_t xrow = 0;
        if (live) xrow = (a.ids ? s_ids[c0 + tok] : first + c0 + tok) / a.rep;
        float acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
        for (int step = lo + warp; step < hi; step += kWarpsMv) {
            const int k = step * kStepK + 32 * t;
            const bool in = k < a.K;
            uint4 c[4][2], sc[2];
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                sc[r] = in ? ld128(scales + (int64_t)(2 * step + (t >> 1)) * lin::kSfTileBytes + 128 * r)
                           : zero;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = row0 + 32 * i + 8 * r + g;
                    c[i][r] = in && row < a.N ? ld128(codes + ((int64_t)row * a.K + k) / 2) : zero;
                }
            }
            Frag<XT> f;
            if (in && live) {
                load_x<XT>(f, a.x, xrow * a.K + k, g);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) f.b[q][i] = 0u;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t s[2][2];  // row half, block
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t word = i == 0 ? sc[r].x : i == 1 ? sc[r].y : i == 2 ? sc[r].z : sc[r].w;
                    const uint32_t two = word >> (16 * (t & 1));
                    s[r][0] = scale_pair<XT>(two & 0xFFu);
                    s[r][1] = scale_pair<XT>((two >> 8) & 0xFFu);
                }
                const uint32_t w0[4] = {c[i][0].x, c[i][0].y, c[i][0].z, c[i][0].w};
                const uint32_t w1[4] = {c[i][1].x, c[i][1].y, c[i][1].z, c[i][1].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t u[4], v[4];
                    unpack<XT>(w0[q], s[0][q >> 1], u);
                    unpack<XT>(w1[q], s[1][q >> 1], v);
                    mma16<XT>(acc[i], u[0], v[0], u[1], v[1], f.b[q][0], f.b[q][1]);
                    mma16<XT>(acc[i], u[2], v[2], u[3], v[3], f.b[q][2], f.b[q][3]);
                }
            }
        }
        // partial sums: column-major, 64 rows a column
        float* mine = s_part[warp];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mine[(2 * t) * kLine + 16 * i + g] = acc[i][0];
            mine[(2 * t + 1) * kLine + 16 * i + g] = acc[i][1];
            mine[(2 * t) * kLine + 16 * i + 8 + g] = acc[i][2];
            mine[(2 * t + 1) * kLine + 16 * i + 8 + g] = acc[i][3];
        }
        __syncthreads();
        for (int idx = tid; idx < ntok * kRows; idx += 32 * kWarpsMv) {
            const int r = idx & (kRows - 1), tk = idx >> 6;
            float v = 0.0f;
#pragma unroll
            for (int p = XT == In::F32 ? 2 : 0; p >= 0; --p) {  // the smallest piece first
                const int at = (XT == In::F32 ? 3 * tk + p : tk) * kLine + r;
#pragma unroll
                for (int w = 0; w < kWarpsMv; ++w) v = fadd(v, s_part[w][at]);
            }
            s_sum[tk * kLine + r] = v;
        }
        lin::tile_sync(S);
        for (int idx = rank * 32 * kWarpsMv + tid; idx < ntok * kRows; idx += S * 32 * kWarpsMv) {
            const int r = idx & (kRows - 1), tk = idx >> 6;
            const int row = row0 + 32 * (r >> 4) + (r & 15);
            float v = s_sum[tk * kLine + r];
            if (S > 1) {
                v = 0.0f;
                for (int k = 0; k < S; ++k) v = fadd(v, ld_cluster(s_sum + tk * kLine + r, k));
            }
            if (row >= a.N) continue;
            v = fmul(v, gb);
            const int64_t p = a.ids ? s_ids[c0 + tk] : first + c0 + tk;
            const int64_t at = p * a.N + row, n_at = (int64_t)e * a.N + row;
            switch (static_cast<Out>(a.out_dt)) {
                case Out::BF16: finish<Out::BF16>(a.ep, v, n_at, at); break;
                case Out::F16: finish<Out::F16>(a.ep, v, n_at, at); break;
                default: finish<Out::F32>(a.ep, v, n_at, at); break;
            }
        }
        lin::tile_sync(S);  // the sums have been read
    }
}

}  // namespace matvec
}  // namespace fos
