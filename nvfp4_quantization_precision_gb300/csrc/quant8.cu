// quant8.cu -- launches of the 8-bit quantization along rows and columns
// (fos_quant8.cuh), by input type and activation, of one tensor and of rows packed
// by group.
#include "fos_quant8.cuh"
#include "fos_ops_launch.cuh"

namespace fos {

namespace {

// sums[g][c]: the rows of `part` that are group g's, added in one order: four
// threads a column take every fourth row each, four loads in flight.
constexpr int kSumCols = 64, kSumParts = 4;
__global__ void __launch_bounds__(kSumCols * kSumParts) k_group_sums(const float* part, const int32_t* bounds,
                                                                     int64_t cols, float* sums) {
    chain_wait();
    chain_release();
    __shared__ float s_sum[kSumParts][kSumCols];
    const int cl = threadIdx.x % kSumCols, sub = threadIdx.x / kSumCols;
    const int64_t c = (int64_t)blockIdx.x * kSumCols + cl;
    const int g = blockIdx.y;
    const int lo = ld_s32(bounds + g), hi = ld_s32(bounds + g + 1);
    float s = 0.0f;
    if (c < cols) {
        for (int p = lo + sub; p < hi; p += 4 * kSumParts) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = p + k * kSumParts < hi ? ld_f32(part + (int64_t)(p + k * kSumParts) * cols + c) : 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) s = fadd(s, v[k]);
        }
    }
    s_sum[sub][cl] = s;
    __syncthreads();
    if (sub == 0 && c < cols) {
        for (int k = 1; k < kSumParts; ++k) s = fadd(s, s_sum[k][cl]);
        sums[g * cols + c] = s;
    }
}

template <In IT, Act A>
cudaError_t go_grouped(const GroupedQuant8Args& b, float* sums, cudaStream_t s) {
    auto k = k_quant8_grouped<IT, A>;
    const size_t smem = kQ8Smem + group_table_bytes(b.G);
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), kQ8Smem + group_table_bytes(kMaxGroups));
    if (e != cudaSuccess) return e;
    const int64_t most = group_tiles_max(b.q.rows, b.G, kQ8Tile) * b.q.tiles_c;
    const int64_t wave = (int64_t)sm_count() *
                         resident_ctas(reinterpret_cast<const void*>(k), smem, kQ8Threads);
    e = launch_chained(k, dim3((unsigned)(most < wave ? most : wave)), kQ8Threads, smem, s, b);
    if (e == cudaSuccess && sums)
        e = launch_chained(k_group_sums, dim3((unsigned)((b.q.cols + kSumCols - 1) / kSumCols), (unsigned)b.G),
                           kSumCols * kSumParts, 0, s, (const float*)b.q.part, (const int32_t*)b.bounds,
                           b.q.cols, sums);
    return e;
}

template <In IT>
cudaError_t grouped_by_act(Act act, const GroupedQuant8Args& b, float* sums, cudaStream_t s) {
    switch (act) {
        case Act::NONE: return go_grouped<IT, Act::NONE>(b, sums, s);
        case Act::RELU: return go_grouped<IT, Act::RELU>(b, sums, s);
        case Act::GELU: return go_grouped<IT, Act::GELU>(b, sums, s);
        case Act::GELU_TANH: return go_grouped<IT, Act::GELU_TANH>(b, sums, s);
        case Act::SILU: return go_grouped<IT, Act::SILU>(b, sums, s);
    }
    return cudaErrorInvalidValue;
}

template <In IT, Act A>
cudaError_t go(const Quant8Args& a, cudaStream_t s) {
    auto k = k_quant8<IT, A>;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), kQ8Smem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (a.rows + kQ8Tile - 1) / kQ8Tile * a.tiles_c;
    Quant8Args b = a;
    b.wave = sm_count() * resident_ctas(reinterpret_cast<const void*>(k), kQ8Smem, kQ8Threads);
    return launch_chained(k, dim3((unsigned)tiles), kQ8Threads, kQ8Smem, s, b);
}

template <In IT>
cudaError_t by_act(Act act, const Quant8Args& a, cudaStream_t s) {
    switch (act) {
        case Act::NONE: return go<IT, Act::NONE>(a, s);
        case Act::RELU: return go<IT, Act::RELU>(a, s);
        case Act::GELU: return go<IT, Act::GELU>(a, s);
        case Act::GELU_TANH: return go<IT, Act::GELU_TANH>(a, s);
        case Act::SILU: return go<IT, Act::SILU>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_quant8(In it, Act act, const Quant8Args& a, cudaStream_t s) {
    switch (it) {
        case In::BF16: return by_act<In::BF16>(act, a, s);
        case In::F16: return by_act<In::F16>(act, a, s);
        case In::F32: return by_act<In::F32>(act, a, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_quant8_grouped(In it, Act act, const GroupedQuant8Args& b, float* sums,
                                  cudaStream_t s) {
    switch (it) {
        case In::BF16: return grouped_by_act<In::BF16>(act, b, sums, s);
        case In::F16: return grouped_by_act<In::F16>(act, b, sums, s);
        case In::F32: return grouped_by_act<In::F32>(act, b, sums, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace fos
