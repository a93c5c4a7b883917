// fos_groups.cuh -- rows packed by group (expert), read from cumulative ends on
// the device: group g has rows [end_{g-1}, end_g), end_g = clamp(offs[g],
// end_{g-1}, rows), and its rows are cut into tiles of kUnit rows that belong to it
// alone (its last one may be short).
//
// The host does not know the ends, so each CTA forms the table of groups itself,
// one warp over at most 1024 ends: entry g holds group g's first row and the
// number of its first tile, entry G the last end and the number of tiles.
#pragma once

#include "fos_block8.cuh"

namespace fos {

struct Group {
    int32_t row, tile;
};
constexpr int kMaxGroups = 1024;  // FOS_LINEAR_MAX_GROUPS
inline __host__ __device__ constexpr size_t group_table_bytes(int G) {
    return ((size_t)(G + 1) * sizeof(Group) + 15) / 16 * 16;
}
// Tiles of `unit` rows that G groups of together `rows` rows can have at most: every
// group with rows adds up to unit - 1 to be a whole number of tiles.
inline __host__ __device__ constexpr int64_t group_tiles_max(int64_t rows, int64_t G, int unit) {
    const int64_t most = G < rows ? G : rows;
    return (rows + most * (unit - 1)) / unit;
}

__device__ __forceinline__ int32_t ld_s32(const int32_t* p) {
    int32_t v;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

namespace lin {

// One value of type OT as it is stored, by a load that stays where it is written: behind
// the wait for the kernel before, and before the same thread's stores (out may be in the
// residual's place).
template <Out OT>
__device__ __forceinline__ uint32_t ld_raw(const void* p, int64_t i) {
    uint32_t v;
    if constexpr (OT == Out::F32)
        asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(static_cast<const float*>(p) + i) : "memory");
    else
        asm volatile("{\n\t.reg .b16 h;\n\tld.global.b16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}"
                     : "=r"(v) : "l"(static_cast<const unsigned short*>(p) + i) : "memory");
    return v;
}
template <Out OT>
__device__ __forceinline__ float raw_value(uint32_t v) {
    if constexpr (OT == Out::F32) return __uint_as_float(v);
    else if constexpr (OT == Out::BF16) return __uint_as_float(v << 16);
    else {
        float f;
        asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(v));
        return f;
    }
}

}  // namespace lin

// The table by one converged warp; lane l takes ceil(G / 32) neighbouring groups.
template <int kUnit>
__device__ __forceinline__ void group_table(Group* t, const int32_t* offs, int G, int32_t rows,
                                            int lane) {
    const int per = (G + 31) >> 5, lo = min(G, lane * per), hi = min(G, lo + per);
    int32_t most = 0;
#pragma unroll 4
    for (int i = lo; i < hi; ++i) {
        most = max(most, ld_s32(offs + i));
        t[i + 1].row = most;
    }
    int32_t before = most;  // largest end of the lanes up to this one
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xFFFFFFFFu, before, d);
        if (lane >= d) before = max(before, o);
    }
    before = __shfl_up_sync(0xFFFFFFFFu, before, 1);
    if (lane == 0) before = 0;
    int32_t row = min(rows, before), tiles = 0;
    for (int i = lo; i < hi; ++i) {
        const int32_t end = min(rows, max(before, t[i + 1].row));
        tiles += (end - row + kUnit - 1) / kUnit;
        t[i + 1] = Group{end, tiles};
        row = end;
    }
    int32_t sum = tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += o;
    }
    sum -= tiles;
    for (int i = lo; i < hi; ++i) t[i + 1].tile += sum;
    if (lane == 0) t[0] = Group{0, 0};
    __syncwarp();
}

// The group of tile `tile` (below t[G].tile): `g`, where the caller's walk stands, or
// the one after it, else by bisection (runs of empty groups).
__host__ __device__ __forceinline__ int group_of(const Group* t, int G, int tile, int g) {
    if (t[g + 1].tile > tile && t[g].tile <= tile) return g;
    if (g + 2 <= G && t[g + 2].tile > tile && t[g + 1].tile <= tile) return g + 1;
    int lo = 0, hi = G;  // t[lo].tile <= tile < t[hi].tile
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t[mid].tile <= tile) lo = mid;
        else hi = mid;
    }
    return lo;
}

}  // namespace fos
