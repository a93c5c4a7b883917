// quant8.cu -- launches of the 8-bit quantization along rows and columns
// (fos_quant8.cuh), by input type and activation.
#include "fos_quant8.cuh"
#include "fos_ops_launch.cuh"

namespace fos {

namespace {

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

}  // namespace fos
