// fos_block8.cuh -- device building blocks of the 8-bit block format the
// feed-forward operators read and write: E4M3 codes with one power-of-two
// (UE8M0) scale per 32 consecutive elements.
//
// The scale of a block with largest magnitude a (NaN dropped) is the smallest
// power of two 2^e, e >= -127, with a <= 448 * 2^e, stored as the byte e + 127;
// a code is E4M3_rn_satfinite(v * 2^-e).  With a = (1 + m / 2^23) * 2^(E - 127)
// and 448 = 1.75 * 2^8 the byte is E - 8, plus one when 1 + m / 2^23 > 1.75,
// and adding 0x1FFFFF to the bits of a carries into the exponent exactly then.
// Multiplying by a power of two is exact, so a code has one rounding.  An
// infinite a gives byte 247, whose inverse scale is still a normal number.
#pragma once

#include "fos_device.cuh"

namespace fos {

// Scale byte of a block with largest magnitude `amax` (>= 0, never NaN).
__device__ __forceinline__ uint32_t scale8_code(float amax) {
    const int e = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 8;
    return (uint32_t)max(e, 0);
}
// 2^-e of a scale byte (0 .. 247), the factor the block's values are multiplied by.
__device__ __forceinline__ float scale8_inv(uint32_t code) {
    return __uint_as_float((254u - code) << 23);
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Four E4M3 codes of two pairs times `inv`, first element in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(uint64_t p0, uint64_t p1, uint64_t inv2) {
    float a, b, c, d;
    upk(mul2(p0, inv2), a, b);
    upk(mul2(p1, inv2), c, d);
    return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// Codes of 16 values (8 pairs).
__device__ __forceinline__ void encode8(const uint64_t (&v)[8], float inv, uint32_t (&w)[4]) {
    const uint64_t inv2 = pk(inv, inv);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = e4m3x4(v[2 * k], v[2 * k + 1], inv2);
}

// One value of data that the kernel before may have written (volatile like load_seg,
// which orders it with the other loads).  Not __ldg: that promises data constant from the
// kernel's start, and this kernel starts while the one before still runs, so the
// compiler may move it past the wait, and L1 may hold its line from before the wait.
// load_seg's lines are not kept in L1; of an output in the place of an input, each
// element's store takes its value from the element's load, and nothing reads it after.
__device__ __forceinline__ float ld_f32(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

// Rounds 16 values to the storage type and stores them.
template <In IT>
__device__ __forceinline__ void store_seg(void* p, const uint64_t (&v)[8]) {
    uint32_t w[InTraits<IT>::kWords];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (IT == In::BF16) {
            w[j] = f32x2_bf16x2(v[j]);
        } else if constexpr (IT == In::F16) {
            w[j] = f32x2_f16x2(v[j]);
        } else {
            float a, b;
            upk(v[j], a, b);
            w[2 * j] = __float_as_uint(a);
            w[2 * j + 1] = __float_as_uint(b);
        }
    }
    st256(p, w);
    if constexpr (IT == In::F32) st256(static_cast<char*>(p) + 32, w + 8);
}

// 16 weights as pairs: fp32, or the data's own type.
template <In IT>
__device__ __forceinline__ void load_weight(const void* w, int64_t elem, bool w32,
                                            uint64_t (&out)[8]) {
    if (w32) {
        Raw<In::F32> r;
        load_seg<In::F32>(r, static_cast<const char*>(w) + elem * 4);
        widen<In::F32>(r, out);
    } else {
        constexpr int64_t kElt = (IT == In::F32) ? 4 : 2;
        Raw<IT> r;
        load_seg<IT>(r, static_cast<const char*>(w) + elem * kElt);
        widen<IT>(r, out);
    }
}

// Address of the scale byte of block (row, j) in either layout; pc4 is the
// number of 4-block tiles per tile-row (tiled), nb the blocks per row (plain).
__device__ __forceinline__ int64_t scale8_at(bool tiled, int64_t row, int64_t j, int64_t nb,
                                             int64_t pc4) {
    return tiled ? tiled_scale_off((int32_t)row, (int32_t)j, (int32_t)pc4) : row * nb + j;
}

// Zeroes the padding of a tiled scale matrix (rows up to the next multiple of
// 128, blocks up to the next multiple of 4), shared over `nthreads` threads.
// It writes no byte of a real scale, so it needs no ordering with the stores
// of those.  Fewer than 127 * 2^24 words of padding rows: 32-bit positions.
__device__ __forceinline__ void clear_tiled_pad(uint8_t* scales, int64_t rows, int64_t nb,
                                                int64_t pc4, uint32_t tid, uint32_t nthreads) {
    const uint32_t t4 = (uint32_t)pc4;
    const uint32_t words = (uint32_t)((rows + 127) / 128 * 128 - rows) * t4;
    for (uint32_t i = tid; i < words; i += nthreads)
        st32(scales + tiled_scale_off((int32_t)(rows + i / t4), (int32_t)(i % t4) * 4, (int32_t)t4),
             0u);
    const int pcol = (int)(pc4 * 4 - nb);
    if (pcol == 0) return;
    for (int64_t r = tid; r < rows; r += nthreads)
        for (int k = 0; k < pcol; ++k)
            st8(scales + tiled_scale_off((int32_t)r, (int32_t)nb + k, (int32_t)t4), 0u);
}

}  // namespace fos
