// norm.cu -- launches of the root-mean-square norm and its backward pass
// (fos_norm.cuh), and the column sums of their partial rows.
#include "fos_norm.cuh"
#include "fos_ops_launch.cuh"

namespace fos {

__global__ void __launch_bounds__(32 * kSumWarps) k_column_sums(const float* part, int64_t parts,
                                                                int64_t cols, float* out) {
    chain_wait();
    chain_release();
    __shared__ float s_sum[kSumWarps][33];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < cols) {
        for (int64_t p = warp; p < parts; p += 8 * kSumWarps) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = p + k * kSumWarps < parts ? ld_f32(part + (p + k * kSumWarps) * cols + c) : 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s = fadd(s, v[k]);
        }
    }
    s_sum[warp][lane] = s;
    __syncthreads();
    // warp w adds the 32 partial sums of column w (a fixed tree)
    float v = s_sum[lane][warp];
    v = lanes_sum<32>(v);
    const int64_t cw = (int64_t)blockIdx.x * 32 + warp;
    if (lane == 0 && cw < cols) out[cw] = v;
}

cudaError_t launch_column_sums(const float* part, int64_t parts, int64_t cols, float* out,
                               cudaStream_t s) {
    return launch_chained(k_column_sums, dim3((unsigned)((cols + 31) / 32)), 32 * kSumWarps, 0, s,
                          part, parts, cols, out);
}

namespace {

// Grid of a row kernel: the resident CTAs, no more than the rows need.
template <class Kernel>
int row_grid(Kernel k, int threads, int64_t rows, int groups) {
    const int64_t full = (int64_t)sm_count() *
                         resident_ctas(reinterpret_cast<const void*>(k), 0, threads);
    const int64_t need = (rows + groups - 1) / groups;
    return (int)(need < full ? need : full);
}

// The same with up to 16 CTAs for the padding rows of tiled scales, which
// would otherwise take a single row's CTA longer than its row.
template <class Kernel>
int norm_grid(Kernel k, int threads, const NormArgs& a, int groups) {
    const int64_t g = row_grid(k, threads, a.rows, groups);
    if (!a.tiled || !a.codes || g >= 16) return (int)g;
    const int64_t words = ((a.rows + 127) / 128 * 128 - a.rows) * a.pc4;
    const int64_t pad = (words + threads - 1) / threads;
    return (int)(g > pad ? g : (pad < 16 ? pad : 16));
}

template <In IT, bool RES, int kT, int kSeg>
cudaError_t norm_go(const NormArgs& a, cudaStream_t s) {
    constexpr int cta = kT < 256 ? 256 : kT;
    auto k = k_rms_norm<IT, RES, kT, kSeg>;
    return launch_chained(k, dim3((unsigned)norm_grid(k, cta, a, cta / kT)), cta, 0, s, a);
}

template <In IT, bool RES>
cudaError_t norm_by_width(const NormArgs& a, cudaStream_t s) {
    // 33.5 M elements, bf16 with a residual, this group and another (us): 512 wide
    // 43.8 and 52.1 (64 threads, half of them idle); 1024 wide 40.9 and 43.9 (32, two
    // segments); 2048 wide 40.5 and 43.0 (64, two); 4096 wide 38.6 and 42.5 (128,
    // two); 8192 wide 38.8 and 40.5 (512, one); 16384 wide 39.1 and 40.9 (1024, one)
    const int64_t nseg = a.cols / 16;
    if (nseg <= 32) return norm_go<IT, RES, 32, 1>(a, s);
    if (nseg <= 64) return norm_go<IT, RES, 64, 1>(a, s);
    if (nseg <= 128) return norm_go<IT, RES, 128, 1>(a, s);
    if (nseg <= 256) return norm_go<IT, RES, 256, 1>(a, s);
    if (nseg <= 512) return norm_go<IT, RES, 256, 2>(a, s);
    if (nseg <= 1024) return norm_go<IT, RES, 512, 2>(a, s);
    auto k = k_rms_norm_wide<IT, RES>;
    return launch_chained(k, dim3((unsigned)row_grid(k, 512, a.rows, 1)), 512, 0, s, a);
}

template <In IT>
cudaError_t norm_by_res(const NormArgs& a, cudaStream_t s) {
    return a.res ? norm_by_width<IT, true>(a, s) : norm_by_width<IT, false>(a, s);
}

template <In IT, int kT, bool DH>
cudaError_t bwd_launch(NormBwdArgs& a, float* dw, float* part, int64_t max_parts, cudaStream_t s) {
    auto k = k_rms_bwd<IT, kT, DH>;
    int64_t grid = row_grid(k, kBwdThreads, a.rows, kBwdThreads / kT);
    if (grid > max_parts) grid = max_parts;
    a.part = !dw ? nullptr : (grid == 1 ? dw : part);  // one CTA writes the result itself
    cudaError_t e = launch_chained(k, dim3((unsigned)grid), kBwdThreads, 0, s, a);
    if (e != cudaSuccess || !dw || grid == 1) return e;
    return launch_column_sums(part, grid, a.cols, dw, s);
}

template <In IT, int kT>
cudaError_t bwd_go(NormBwdArgs& a, float* dw, float* part, int64_t max_parts, cudaStream_t s) {
    return a.dh ? bwd_launch<IT, kT, true>(a, dw, part, max_parts, s)
                : bwd_launch<IT, kT, false>(a, dw, part, max_parts, s);
}

template <In IT>
cudaError_t bwd_by_width(NormBwdArgs& a, float* dw, float* part, int64_t max_parts,
                         cudaStream_t s) {
    const int64_t nseg = a.cols / 16;
    if (nseg <= 32) return bwd_go<IT, 32>(a, dw, part, max_parts, s);
    if (nseg <= 64) return bwd_go<IT, 64>(a, dw, part, max_parts, s);
    if (nseg <= 128) return bwd_go<IT, 128>(a, dw, part, max_parts, s);
    if (nseg <= 256) return bwd_go<IT, 256>(a, dw, part, max_parts, s);
    if (nseg <= 512) return bwd_go<IT, 512>(a, dw, part, max_parts, s);
    auto k = k_rms_bwd_wide<IT>;
    auto input_grad = [&] {
        return launch_chained(k, dim3((unsigned)row_grid(k, 512, a.rows, 1)), 512, 0, s, a);
    };
    if (!dw) return input_grad();
    const int64_t strips = (a.cols + 4095) / 4096;
    int64_t parts = (2 * sm_count() + strips - 1) / strips;
    if (parts > a.rows) parts = a.rows;
    if (parts > max_parts) parts = max_parts;
    a.part = parts == 1 ? dw : part;
    auto weight_grad = [&] {
        return launch_chained(k_rms_dw_wide<IT>, dim3((unsigned)strips, (unsigned)parts), 256, 0, s, a);
    };
    // the weight gradient reads dy and h as well, so it goes first where dx takes
    // their place (2048 x 16384 bf16 with dh: 90.7 us, the other way 88.1)
    const bool replaced = a.dx == a.dy || a.dx == a.h;
    cudaError_t e = replaced ? weight_grad() : input_grad();
    if (e == cudaSuccess) e = replaced ? input_grad() : weight_grad();
    if (e != cudaSuccess || parts == 1) return e;
    return launch_column_sums(part, parts, a.cols, dw, s);
}

}  // namespace

cudaError_t launch_rms_norm(In it, const NormArgs& a, cudaStream_t s) {
    switch (it) {
        case In::BF16: return norm_by_res<In::BF16>(a, s);
        case In::F16: return norm_by_res<In::F16>(a, s);
        case In::F32: return norm_by_res<In::F32>(a, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_rms_bwd(In it, NormBwdArgs a, float* dw, float* part, int64_t max_parts,
                           cudaStream_t s) {
    switch (it) {
        case In::BF16: return bwd_by_width<In::BF16>(a, dw, part, max_parts, s);
        case In::F16: return bwd_by_width<In::F16>(a, dw, part, max_parts, s);
        case In::F32: return bwd_by_width<In::F32>(a, dw, part, max_parts, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace fos
