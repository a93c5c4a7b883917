// fos_ops_api.cu -- host side of the feed-forward operators' entry points
// (fos_rms_norm ... fos_linear4 in include/fos.h): every argument is checked
// before the CUDA runtime is touched, the data's device is made current for
// the call, nothing is allocated and the host is not synchronised.
#include <cmath>
#include <cstdint>

#include "../../include/fos.h"
#include "fos_act.cuh"
#include "fos_host.cuh"
#include "fos_linear.cuh"
#include "fos_norm.cuh"
#include "fos_ops_launch.cuh"
#include "fos_quant8.cuh"

using namespace fos;

namespace {

bool valid_layout(int l) { return l == FOS_SCALES_PLAIN || l == FOS_SCALES_TILED; }
bool valid_act(int a) { return a >= FOS_ACT_NONE && a <= FOS_ACT_SILU; }

// Sizes of an 8-bit block-scaled tensor: whole 32-element blocks, positions
// that fit the kernels' 32-bit row and block numbers.
fos_status check_shape8(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return FOS_ERR_INVALID_ARG;
    if (cols % 32 != 0) return FOS_ERR_UNSUPPORTED;
    if (rows >= (INT64_C(1) << 30) || cols >= (INT64_C(1) << 30)) return FOS_ERR_UNSUPPORTED;
    if (cols > 0 && rows > (INT64_C(1) << 40) / cols) return FOS_ERR_UNSUPPORTED;
    return FOS_OK;
}

int64_t pc4_of(int64_t cols) { return (cols / 32 + 3) / 4; }

// A codes / scales pair: both or neither; codes aligned to `ca`, tiled scales
// to whole words.
fos_status check_pair(const uint8_t* codes, const uint8_t* scales, uintptr_t ca, bool tiled) {
    if (!codes != !scales) return FOS_ERR_INVALID_ARG;
    if (codes && (!aligned(codes, ca) || (tiled && !aligned(scales, 4)))) return FOS_ERR_MISALIGNED;
    return FOS_OK;
}

// One device for every pointer that is given; the first must be.
int device_of_given(std::initializer_list<const void*> ptrs) {
    int dev = -1;
    for (const void* p : ptrs) {
        if (!p) continue;
        const int d = device_of(p);
        if (d < 0 || (dev >= 0 && d != dev)) return -1;
        dev = d;
    }
    return dev;
}

// One tensor of a call.  An output (`may` given) may not touch another tensor, but
// for the inputs named in `may` (a bit each, by position in the list), whose place
// it may take whole: there each element is read before the one thread that reads
// it writes it.
struct Region {
    const void* p;
    int64_t bytes;
    int may = -1;  // -1: an input
};

// Whether the outputs of a call keep apart from its other tensors.
bool keep_apart(std::initializer_list<Region> all) {
    const Region* r = all.begin();
    const int n = (int)all.size();
    for (int i = 0; i < n; ++i) {
        if (r[i].may < 0 || !r[i].p || r[i].bytes <= 0) continue;
        const uintptr_t a = reinterpret_cast<uintptr_t>(r[i].p), a1 = a + (uintptr_t)r[i].bytes;
        for (int j = 0; j < n; ++j) {
            if (j == i || !r[j].p || r[j].bytes <= 0 || (r[j].may >= 0 && j < i)) continue;
            const uintptr_t b = reinterpret_cast<uintptr_t>(r[j].p), b1 = b + (uintptr_t)r[j].bytes;
            if (a >= b1 || b >= a1) continue;
            const bool place = r[j].may < 0 && (r[i].may >> j & 1) && a == b && a1 == b1;
            if (!place) return false;
        }
    }
    return true;
}

int64_t elt_of(int dt) { return dt == FOS_FP32 ? 4 : 2; }

cudaStream_t stream_of(fos_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

int64_t q8_tiles(int64_t rows) { return (rows + kQ8Tile - 1) / kQ8Tile; }

fos_status run_quant8(const void* x, const void* pre, fos_dtype dt, int64_t rows, int64_t cols,
                      int act, int layout, void* d, uint8_t* codes, uint8_t* scales,
                      uint8_t* codes_t, uint8_t* scales_t, float* dbias, void* workspace,
                      size_t workspace_bytes, cudaStream_t s) {
    if (!valid_dtype(dt) || !valid_layout(layout) || !valid_act(act)) return FOS_ERR_INVALID_ARG;
    fos_status st = check_shape8(rows, cols);
    if (st) return st;
    if (cols == 0) return FOS_OK;
    if (rows > 0 && !d && !codes && !scales && !codes_t && !scales_t && !dbias)
        return FOS_ERR_INVALID_ARG;
    if (rows > 0 && (!x || (act != FOS_ACT_NONE && !pre))) return FOS_ERR_INVALID_ARG;
    if (!aligned(x, 32) || !aligned(pre, 32) || !aligned(d, 32) || !aligned(dbias, 4))
        return FOS_ERR_MISALIGNED;
    const bool tiled = layout == FOS_SCALES_TILED;
    st = check_pair(codes, scales, 16, tiled);
    if (st) return st;
    st = check_pair(codes_t, scales_t, 32, tiled);
    if (st) return st;
    const int64_t tiles_r = q8_tiles(rows), tiles_c = (cols + kQ8Tile - 1) / kQ8Tile;
    if (tiles_r > INT64_C(0x7FFFFFFF) / tiles_c) return FOS_ERR_UNSUPPORTED;
    const bool sums = dbias && tiles_r > 1;
    if (sums) {
        if (!workspace || workspace_bytes < fos_act_backward_workspace_bytes(rows, cols))
            return FOS_ERR_INVALID_ARG;
        if (!aligned(workspace, 256)) return FOS_ERR_MISALIGNED;
    }
    if (rows == 0 && !dbias) return FOS_OK;
    const int64_t nb = rows * cols * elt_of(dt), rows_pad = (rows + 31) / 32 * 32;
    if (!keep_apart({{x, nb}, {act != FOS_ACT_NONE ? pre : nullptr, nb}, {d, nb, 3},
                     {codes, rows * cols, 0}, {scales, fos_scales8_bytes(rows, cols, layout), 0},
                     {codes_t, cols * rows_pad, 0},
                     {scales_t, codes_t ? fos_scales8_bytes(cols, rows_pad, layout) : 0, 0},
                     {dbias, cols * 4, 0},
                     {sums ? workspace : nullptr,
                      (int64_t)fos_act_backward_workspace_bytes(rows, cols), 0}}))
        return FOS_ERR_INVALID_ARG;
    const int dev = device_of_given({x, act != FOS_ACT_NONE ? pre : nullptr, d, codes, scales,
                                     codes_t, scales_t, dbias, sums ? workspace : nullptr});
    if (dev < 0) return FOS_ERR_INVALID_ARG;
    DeviceScope scope(dev);
    if (scope.st) return scope.st;
    if (rows == 0) return cuda_status(cudaMemsetAsync(dbias, 0, sizeof(float) * cols, s));
    Quant8Args a{};
    a.x = x;
    a.pre = pre;
    a.d = d;
    a.codes = codes;
    a.scales = scales;
    a.codes_t = codes_t;
    a.scales_t = scales_t;
    a.part = dbias ? (sums ? static_cast<float*>(workspace) : dbias) : nullptr;
    a.rows = rows;
    a.cols = cols;
    a.rows_pad = rows_pad;
    a.tiles_c = tiles_c;
    a.pc4 = pc4_of(cols);
    a.pc4_t = pc4_of(a.rows_pad);
    a.tiled = tiled;
    cudaError_t e = launch_quant8(in_of(dt), static_cast<Act>(act), a, s);
    if (e == cudaSuccess && sums) e = launch_column_sums(a.part, tiles_r, cols, dbias, s);
    return cuda_status(e);
}

fos_status run_linear(LinearCall c, const fos_epilogue* e, void* out, cudaStream_t s) {
    if (!e || !valid_dtype(e->out_dt) || !valid_act(e->act) ||
        (e->bias && e->bias_dt != FOS_FP32 && e->bias_dt != e->out_dt))
        return FOS_ERR_INVALID_ARG;
    if (c.M < 0 || c.N < 0 || c.K < 0) return FOS_ERR_INVALID_ARG;
    if (c.N % 16 || c.K % 32 || c.K == 0) return FOS_ERR_UNSUPPORTED;
    if (c.M >= (INT64_C(1) << 30) || c.N >= (INT64_C(1) << 30) || c.K >= (INT64_C(1) << 30) ||
        (c.N > 0 && c.M > (INT64_C(1) << 40) / c.N) || c.M > (INT64_C(1) << 40) / c.K ||
        c.N > (INT64_C(1) << 40) / c.K)
        return FOS_ERR_UNSUPPORTED;
    if (c.M == 0 || c.N == 0) return FOS_OK;
    if (!c.a || !c.as || !c.b || !c.bs || !out || (c.fmt4 && (!c.ep.a_amax || !c.ep.b_amax)))
        return FOS_ERR_INVALID_ARG;
    if (!aligned(c.a, 16) || !aligned(c.as, 16) || !aligned(c.b, 16) || !aligned(c.bs, 16) ||
        !aligned(out, 16) || !aligned(e->residual, 16) || !aligned(e->pre, 16) ||
        !aligned(e->bias, 16))
        return FOS_ERR_MISALIGNED;
    const int64_t blk = c.fmt4 ? 16 : 32, half = c.fmt4 ? 2 : 1, no = c.M * c.N * elt_of(e->out_dt);
    auto tiles = [&](int64_t rows) { return (rows + 127) / 128 * ((c.K + 4 * blk - 1) / (4 * blk)) * 512; };
    if (!keep_apart({{e->residual, no}, {c.a, c.M * c.K / half}, {c.as, tiles(c.M)},
                     {c.b, c.N * c.K / half}, {c.bs, tiles(c.N)},
                     {c.ep.a_amax, 4 * (c.ep.a_row ? c.M : 1)}, {c.ep.b_amax, 4},
                     {e->bias, c.N * elt_of(e->bias_dt)}, {out, no, 1}, {e->pre, no, 0}}))
        return FOS_ERR_INVALID_ARG;
    const int dev = device_of_given({c.a, c.as, c.b, c.bs, c.ep.a_amax, c.ep.b_amax, e->bias,
                                     e->residual, e->pre, out});
    if (dev < 0) return FOS_ERR_INVALID_ARG;
    DeviceScope scope(dev);
    if (scope.st) return scope.st;
    c.ep.bias = e->bias;
    c.ep.bias32 = e->bias_dt == FOS_FP32;
    c.ep.residual = e->residual;
    c.ep.pre = e->pre;
    c.ep.out = out;
    c.ep.act = e->act;
    c.out = in_of(static_cast<fos_dtype>(e->out_dt));
    return cuda_status(launch_linear(c, s));
}

}  // namespace

extern "C" {

int64_t fos_scales8_bytes(int64_t rows, int64_t cols, int scale_layout) {
    // of a column-wise form too, whose rows padded to 32 may reach 2^30
    if (rows < 0 || cols < 0 || cols % 32 != 0 || !valid_layout(scale_layout)) return -1;
    if (rows > (INT64_C(1) << 30) || cols > (INT64_C(1) << 30)) return -1;
    if (scale_layout == FOS_SCALES_PLAIN) return rows * (cols / 32);
    return (rows + 127) / 128 * 128 * (pc4_of(cols) * 4);
}

fos_status fos_rms_norm(const void* x, const void* residual, const void* weight, fos_dtype dt,
                        fos_dtype weight_dt, int64_t rows, int64_t cols, float eps,
                        int scale_layout, void* h, void* y, uint8_t* codes, uint8_t* scales,
                        float* rstd, fos_stream_t stream) {
    if (!valid_dtype(dt) || (weight_dt != FOS_FP32 && weight_dt != dt) ||
        !valid_layout(scale_layout) || !(eps >= 0.0f) || std::isinf(eps))
        return FOS_ERR_INVALID_ARG;
    fos_status st = check_shape8(rows, cols);
    if (st) return st;
    if (rows == 0) return FOS_OK;
    if (cols == 0) return FOS_ERR_UNSUPPORTED;
    if (!x || !weight || (!h && !y && !codes && !scales && !rstd)) return FOS_ERR_INVALID_ARG;
    if (!aligned(x, 32) || !aligned(residual, 32) || !aligned(weight, 32) || !aligned(h, 32) ||
        !aligned(y, 32) || !aligned(rstd, 4))
        return FOS_ERR_MISALIGNED;
    st = check_pair(codes, scales, 16, scale_layout == FOS_SCALES_TILED);
    if (st) return st;
    const int64_t nb = rows * cols * elt_of(dt);
    if (!keep_apart({{x, nb}, {residual, nb}, {weight, cols * elt_of(weight_dt)}, {h, nb, 3}, {y, nb, 0},
                     {codes, rows * cols, 0}, {scales, fos_scales8_bytes(rows, cols, scale_layout), 0},
                     {rstd, rows * 4, 0}}))
        return FOS_ERR_INVALID_ARG;
    const int dev = device_of_given({x, residual, weight, h, y, codes, scales, rstd});
    if (dev < 0) return FOS_ERR_INVALID_ARG;
    DeviceScope scope(dev);
    if (scope.st) return scope.st;
    NormArgs a{};
    a.x = x;
    a.res = residual;
    a.w = weight;
    a.h = h;
    a.y = y;
    a.codes = codes;
    a.scales = scales;
    a.rstd = rstd;
    a.rows = rows;
    a.cols = cols;
    a.pc4 = pc4_of(cols);
    a.inv_cols = 1.0f / (float)cols;
    a.inv_cols_lo = (float)(1.0 / (double)cols - (double)a.inv_cols);
    a.eps = eps;
    a.w32 = weight_dt == FOS_FP32;
    a.tiled = scale_layout == FOS_SCALES_TILED;
    return cuda_status(launch_rms_norm(in_of(dt), a, stream_of(stream)));
}

size_t fos_rms_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows <= 1 || cols <= 0 || check_shape8(rows, cols)) return 0;
    return (size_t)(rows < kMaxParts ? rows : kMaxParts) * (size_t)cols * sizeof(float);
}

fos_status fos_rms_norm_backward(const void* dy, const void* h, const void* dh, const float* rstd,
                                 const void* weight, fos_dtype dt, fos_dtype weight_dt,
                                 int64_t rows, int64_t cols, void* dx, float* dweight,
                                 void* workspace, size_t workspace_bytes, fos_stream_t stream) {
    if (!valid_dtype(dt) || (weight_dt != FOS_FP32 && weight_dt != dt)) return FOS_ERR_INVALID_ARG;
    fos_status st = check_shape8(rows, cols);
    if (st) return st;
    if (cols == 0) return rows == 0 ? FOS_OK : FOS_ERR_UNSUPPORTED;
    if (rows == 0 && !dweight) return FOS_OK;
    if (rows > 0 && (!dy || !h || !rstd || !weight || !dx)) return FOS_ERR_INVALID_ARG;
    if (!aligned(dy, 32) || !aligned(h, 32) || !aligned(dh, 32) || !aligned(weight, 32) ||
        !aligned(dx, 32) || !aligned(dweight, 32) || !aligned(rstd, 4))
        return FOS_ERR_MISALIGNED;
    const size_t need = dweight ? fos_rms_norm_backward_workspace_bytes(rows, cols) : 0;
    if (need) {
        if (!workspace || workspace_bytes < need) return FOS_ERR_INVALID_ARG;
        if (!aligned(workspace, 256)) return FOS_ERR_MISALIGNED;
    }
    const int64_t nb = rows * cols * elt_of(dt);
    if (!keep_apart({{dy, nb}, {h, nb}, {dh, nb}, {rstd, rows * 4}, {weight, cols * elt_of(weight_dt)},
                     {dx, nb, 7}, {dweight, cols * 4, 0}, {need ? workspace : nullptr, (int64_t)need, 0}}))
        return FOS_ERR_INVALID_ARG;
    const int dev = rows > 0 ? device_of_given({dy, h, dh, rstd, weight, dx, dweight,
                                                need ? workspace : nullptr})
                             : device_of(dweight);
    if (dev < 0) return FOS_ERR_INVALID_ARG;
    DeviceScope scope(dev);
    if (scope.st) return scope.st;
    cudaStream_t s = stream_of(stream);
    if (rows == 0) return cuda_status(cudaMemsetAsync(dweight, 0, sizeof(float) * cols, s));
    NormBwdArgs a{};
    a.dy = dy;
    a.h = h;
    a.dh = dh;
    a.rstd = rstd;
    a.w = weight;
    a.dx = dx;
    a.rows = rows;
    a.cols = cols;
    a.inv_cols = 1.0f / (float)cols;
    a.inv_cols_lo = (float)(1.0 / (double)cols - (double)a.inv_cols);
    a.w32 = weight_dt == FOS_FP32;
    return cuda_status(launch_rms_bwd(in_of(dt), a, dweight, static_cast<float*>(workspace),
                                      rows < kMaxParts ? rows : kMaxParts, s));
}

fos_status fos_quantize8(const void* x, fos_dtype dt, int64_t rows, int64_t cols, int scale_layout,
                         uint8_t* codes, uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t,
                         fos_stream_t stream) {
    return run_quant8(x, nullptr, dt, rows, cols, FOS_ACT_NONE, scale_layout, nullptr, codes, scales,
                      codes_t, scales_t, nullptr, nullptr, 0, stream_of(stream));
}

size_t fos_act_backward_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows <= kQ8Tile || cols <= 0 || check_shape8(rows, cols)) return 0;
    return (size_t)q8_tiles(rows) * (size_t)cols * sizeof(float);
}

fos_status fos_act_backward(const void* dout, const void* pre, fos_dtype dt, int64_t rows,
                            int64_t cols, int act, int scale_layout, void* d, uint8_t* codes,
                            uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, float* dbias,
                            void* workspace, size_t workspace_bytes, fos_stream_t stream) {
    return run_quant8(dout, pre, dt, rows, cols, act, scale_layout, d, codes, scales, codes_t,
                      scales_t, dbias, workspace, workspace_bytes, stream_of(stream));
}

fos_status fos_linear8(const uint8_t* a_codes, const uint8_t* a_scales_tiled,
                       const uint8_t* b_codes, const uint8_t* b_scales_tiled, int64_t M, int64_t N,
                       int64_t K, const fos_epilogue* epilogue, void* out, fos_stream_t stream) {
    LinearCall c{};
    c.a = a_codes;
    c.as = a_scales_tiled;
    c.b = b_codes;
    c.bs = b_scales_tiled;
    c.M = M;
    c.N = N;
    c.K = K;
    return run_linear(c, epilogue, out, stream_of(stream));
}

fos_status fos_linear4(const uint8_t* a_codes, const uint8_t* a_scales_tiled, const float* a_amax,
                       const uint8_t* b_codes, const uint8_t* b_scales_tiled, const float* b_amax,
                       int64_t M, int64_t N, int64_t K, const fos_config* cfg,
                       const fos_epilogue* epilogue, void* out, fos_stream_t stream) {
    if (!cfg || (cfg->granularity != FOS_SCALE_TENSOR && cfg->granularity != FOS_SCALE_ROW))
        return FOS_ERR_INVALID_ARG;
    if (cfg->block != FOS_BLOCK_1X16 || (cfg->e4m3_bound != 448 && cfg->e4m3_bound != 256))
        return FOS_ERR_UNSUPPORTED;
    LinearCall c{};
    c.a = a_codes;
    c.as = a_scales_tiled;
    c.b = b_codes;
    c.bs = b_scales_tiled;
    c.M = M;
    c.N = N;
    c.K = K;
    c.fmt4 = true;
    c.ep.a_amax = a_amax;
    c.ep.b_amax = b_amax;
    c.ep.a_row = cfg->granularity == FOS_SCALE_ROW;
    c.ep.six_bound = 6.0f * (float)cfg->e4m3_bound;
    return run_linear(c, epilogue, out, stream_of(stream));
}

}  // extern "C"
