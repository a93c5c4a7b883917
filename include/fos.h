/*
 * fos.h -- C ABI of the GB300 (sm_103a) NVFP4 four-over-six block quantizer.
 *
 * The method (torchao PR "Add the four-over-six grouped GEMM and dispatcher
 * wiring", description and first commit): every quantization block -- 1x16
 * elements along a row, or a 16x16 tile for weights -- is encoded twice under
 * an FP32 global scale, once as standard NVFP4 (block amax mapped to E2M1
 * value 6 by an E4M3 block scale) and once as a 1.5x-scale candidate (block
 * amax mapped to 4).  Both are rounded to E2M1 with correctly-rounded FP32
 * division, decoded exactly, and compared by MAE or MSE; the lower-error
 * candidate's packed E2M1 codes and E4M3 scale are stored (torchao PR "Add a
 * CuTe DSL fast-path kernel for four-over-six quantize": pinned rounding,
 * pinned width-16 error reduction, NaN-dropping block amax, NaN -> +6).
 *
 * Conventions shared by every entry point
 *   - Data pointers (x, out, codes, scales, amax, offs, workspaces) are
 *     DEVICE pointers owned by the caller; the library never allocates, frees
 *     or keeps them (fos_qdq_fused_static uses one fixed array of its
 *     own).  Host-side arrays (the pointer / size lists of the list calls)
 *     are read during the call only.
 *   - Tensors are row-major and contiguous: x is [rows, cols]; codes are
 *     [rows, cols/2] bytes, element 2j in the low nibble of byte j; scales are
 *     E4M3 bytes [rows, cols/16] (1x16) or [rows/16, cols/16] (16x16), plain
 *     row-major (fos_swizzle_scales gives the tiled GEMM layout).
 *   - cols % 16 == 0; with 16x16 blocks also rows % 16 == 0.
 *   - x / out must be 32-byte aligned, codes 8-byte aligned (any row slice of
 *     a tensor from the CUDA caching allocator satisfies this).
 *   - Work is enqueued on `stream` of the device that owns the data and the
 *     call returns without synchronising the host (fos_workspace_error and
 *     fos_tile_amax_status, which read a result back, are the exceptions).  The caller's current device is
 *     restored before return.
 *   - Every argument is validated on the host before anything is launched;
 *     a failed check returns an error status and launches nothing.  CUDA
 *     launch failures return FOS_ERR_CUDA.  Kernels never trap.  The only
 *     waits on other work are the bounded ones of fos_qdq_fused (between the
 *     CTAs of its cooperative launch) and of the column-wise kernel (on its
 *     own TMA loads); each gives up after about a second and reports it, so
 *     no call can hang the device.
 *   - Global scale (reading of "FP32 global scale"): S = (6 * bound) / A,
 *     correctly rounded, for a global amax A; S = 1 when A is zero, negative,
 *     NaN or Inf; S = FLT_MAX when the quotient overflows.
 */
#ifndef FOS_H
#define FOS_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FOS_API __attribute__((visibility("default")))
#else
#define FOS_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Identical to cudaStream_t; 0 is the legacy default stream. */
typedef struct CUstream_st* fos_stream_t;

typedef enum {
    FOS_OK = 0,
    FOS_ERR_INVALID_ARG = 1, /* null pointer, negative size, bad enum value   */
    FOS_ERR_UNSUPPORTED = 2, /* shape / knob / dtype combination not offered  */
    FOS_ERR_MISALIGNED = 3,  /* pointer alignment rule above violated         */
    FOS_ERR_CUDA = 4,        /* a CUDA runtime call or launch failed          */
    FOS_ERR_NONUNIFORM_TILE_AMAX = 5 /* fos_tile_amax_status: a 16-row tile's
                                        per-row amax entries differ         */
} fos_status;

typedef enum { FOS_BF16 = 0, FOS_FP16 = 1, FOS_FP32 = 2 } fos_dtype;

enum { FOS_BLOCK_1X16 = 0, FOS_BLOCK_16X16 = 1 };
enum { FOS_MODE_STANDARD = 0, FOS_MODE_4OVER6 = 1 };
enum { FOS_MAE = 0, FOS_MSE = 1 };
enum { FOS_ERR_EXACT_F32 = 0, FOS_ERR_F16 = 1 };
enum { FOS_SCALE_TENSOR = 0, FOS_SCALE_ROW = 1 };
enum { FOS_ORDER_TREE = 0, FOS_ORDER_SEQ = 1 };
enum { FOS_SCALES_PLAIN = 0, FOS_SCALES_TILED = 1 };

/* The knobs the pages name (Megatron PR "Fuse NVFP4 fake-QAT quantize-
 * dequantize with CuTe DSL", numerical contract: standard NVFP4 plus 4over6
 * MAE/MSE, E4M3 256/448, exact-error / FP16-error; torchao PRs: 1x16 / 16x16
 * blocks, per-tensor or row-scaled global scale). */
typedef struct {
    int block;         /* FOS_BLOCK_1X16 | FOS_BLOCK_16X16                       */
    int mode;          /* FOS_MODE_STANDARD (map-to-6 only) | FOS_MODE_4OVER6    */
    int err_metric;    /* FOS_MAE | FOS_MSE                     (4over6 only)    */
    int err_precision; /* FOS_ERR_EXACT_F32 | FOS_ERR_F16       (4over6 only)    */
    int e4m3_bound;    /* 448 | 256: E4M3 value the global scale maps the amax to */
    int granularity;   /* FOS_SCALE_TENSOR | FOS_SCALE_ROW                       */
    int amax_is_input; /* 1: caller supplies amax; 0: library computes, writes it */
    int err_order;     /* how a block's 16 error terms are summed (4over6 only):
                        * FOS_ORDER_TREE (0): the pinned width-16 tree of the
                        *   torchao fast-path PR, for w = 8,4,2,1: t[i] += t[i+w];
                        * FOS_ORDER_SEQ (1): in element order, t0 + t1 + ... + t15
                        *   (the Transformer Engine term order the Megatron PR
                        *   keeps, "Packed pair arithmetic"); 1x16 blocks only,
                        *   FOS_ERR_UNSUPPORTED with 16x16 in 4over6 mode.     */
    int scale_layout;  /* where the quantize calls write the E4M3 block scales:
                        * FOS_SCALES_PLAIN (0): row-major [rows, cols/16]
                        *   ([rows/16, cols/16] for 16x16);
                        * FOS_SCALES_TILED (1): straight into the tiled layout
                        *   of block-scaled FP4 GEMMs that fos_swizzle_scales
                        *   produces (fos_swizzled_scales_bytes(rows, cols)
                        *   bytes, zero padding included), ready for fos_mm;
                        *   1x16 blocks and fewer than 2^30 rows (of x, and
                        *   of x^T for fos_quantize_colwise) only, else
                        *   FOS_ERR_UNSUPPORTED (fos_quantize, fos_quantize_list,
                        *   fos_quantize_overlap, fos_quantize_colwise); the
                        *   grouped quantize and fos_dequantize take plain
                        *   scales only and return FOS_ERR_UNSUPPORTED.     */
} fos_config;

/*
 * fos_amax -- global amax pass (Megatron PR, fused data path: FP32
 * per-tensor amax computed before the fused kernel).  NaN-dropping max|x|
 * with initial +0: a NaN never becomes the amax and an all-NaN or empty
 * scope gives 0.
 *   granularity FOS_SCALE_TENSOR: amax[0] = over all of x.
 *   granularity FOS_SCALE_ROW:    amax[r] = over row r, r < rows.
 * Errors: FOS_ERR_INVALID_ARG (null pointers with nonzero size, negative
 * sizes, bad enum), FOS_ERR_UNSUPPORTED (cols % 16 != 0), FOS_ERR_MISALIGNED.
 */
FOS_API fos_status fos_amax(const void* x, fos_dtype dt, int64_t rows, int64_t cols, int granularity,
                    float* amax, fos_stream_t stream);

/*
 * fos_quantize -- four-over-six (or standard) NVFP4 quantize of x [rows, cols]
 * of dtype bf16, fp16 or fp32 (torchao fast-path PR: the quantizer op;
 * grouped PR: per-tensor or row-scaled global scale, 1x16 / 16x16 blocks).
 *   amax   [1] (FOS_SCALE_TENSOR) or [rows] (FOS_SCALE_ROW): read when
 *          cfg->amax_is_input, otherwise computed first and written.
 *          With 16x16 blocks and FOS_SCALE_ROW the per-row amax must be
 *          uniform inside each 16-row tile (grouped PR, tile-uniform
 *          contract); each tile uses the amax of its first row.
 *   codes  [rows, cols/2] out; scales out (layout above).
 * Errors as for fos_amax, plus FOS_ERR_UNSUPPORTED for a bad bound, block,
 * mode or (16x16) rows % 16 != 0.
 */
FOS_API fos_status fos_quantize(const void* x, fos_dtype dt, int64_t rows, int64_t cols,
                        const fos_config* cfg, float* amax, uint8_t* codes, uint8_t* scales,
                        fos_stream_t stream);

/*
 * fos_check_tile_amax -- validation of the tile-uniform contract above
 * (grouped PR: with 16x16 blocks a row-scaled global scale must be the same
 * for the 16 rows of a tile, so the per-row amax must be): counts the 16-row
 * tiles of amax [rows] whose 16 entries are not all bitwise equal and writes
 * the count to *bad (device int64, cleared by the call).  rows % 16 == 0;
 * amax 4-byte aligned.  Asynchronous like every call; fos_quantize itself
 * never checks (it uses each tile's first-row amax), so a caller that wants
 * the check runs this first.  Errors: FOS_ERR_INVALID_ARG (null pointer with
 * rows > 0, negative rows), FOS_ERR_UNSUPPORTED (rows % 16 != 0),
 * FOS_ERR_MISALIGNED.
 */
FOS_API fos_status fos_check_tile_amax(const float* amax, int64_t rows, int64_t* bad,
                                       fos_stream_t stream);

/*
 * fos_tile_amax_status -- the validating read of that count: waits for
 * `stream`, reads *bad and returns FOS_OK when it is zero and
 * FOS_ERR_NONUNIFORM_TILE_AMAX otherwise (FOS_ERR_INVALID_ARG for a pointer
 * that is not device memory, FOS_ERR_CUDA when the wait fails).  This call
 * synchronises the host.
 */
FOS_API fos_status fos_tile_amax_status(const int64_t* bad, fos_stream_t stream);

/*
 * fos_quantize_list -- fos_quantize over a list of n tensors of one dtype
 * and one configuration; entry i reads x[i] (rows[i] x cols[i]) and writes
 * amax[i], codes[i], scales[i] exactly as fos_quantize would.  With 1x16
 * blocks, per-tensor scale and the amax computed by the library, the work is
 * pipelined: the launch that encodes tensor i also runs the amax pass of
 * tensor i+1 (every warp loads its next-tensor segment before encoding and
 * folds it into its max afterwards; the encode is bound by instruction
 * issue, the amax pass by HBM reads), so a list costs about one amax pass
 * plus n encodes.  Other configurations run the entries one after another.
 * Host arrays must hold n entries; errors as for fos_quantize (the first
 * failing entry's status, nothing launched).
 */
FOS_API fos_status fos_quantize_list(int n, const void* const* x, fos_dtype dt,
                                     const int64_t* rows, const int64_t* cols,
                                     const fos_config* cfg, float* const* amax,
                                     uint8_t* const* codes, uint8_t* const* scales,
                                     fos_stream_t stream);

/*
 * fos_quantize_overlap -- one stage of the list pipeline, for callers that
 * pipeline their own tensors: quantize x (1x16 blocks, per-tensor scale,
 * cfg->amax_is_input must be 1, amax given) and, in the same launch, compute
 * the per-tensor amax of x_next (same dtype, rows_next x cols_next) into
 * amax_next[0] (cleared first, written by the launch).  With amax_next NULL
 * it is fos_quantize.  Returns FOS_ERR_UNSUPPORTED for other configurations.
 */
FOS_API fos_status fos_quantize_overlap(const void* x, fos_dtype dt, int64_t rows, int64_t cols,
                                        const fos_config* cfg, const float* amax,
                                        uint8_t* codes, uint8_t* scales, const void* x_next,
                                        int64_t rows_next, int64_t cols_next,
                                        float* amax_next, fos_stream_t stream);

/*
 * fos_quantize_colwise -- the column-wise operand: fos_quantize applied to
 * x^T ([cols, rows]), computed from the row-major x [rows, cols] without
 * forming x^T.  Blocks are 16 consecutive rows of one column of x:
 *   codes_t [cols, rows/2], scales_t [cols, rows/16] (row c of x^T = column
 *   c of x, low nibble = the upper of two rows).
 * With codes and scales both non-NULL the row-wise result of x ([rows,
 * cols/2], [rows, cols/16], exactly fos_quantize's) is written by the same
 * launch from the same read of x; both NULL skips it.  1x16 blocks and a
 * per-tensor scale only (the amax of x and of x^T are the same value);
 * rows % 16 == 0 and cols % 16 == 0.  amax as in fos_quantize.  The pages
 * list transpose / column-wise output as a non-goal of their QDQ path (the
 * Megatron PR's deliberate non-goals); this is the layout a weight-gradient
 * GEMM reads, built with the same arithmetic.
 */
FOS_API fos_status fos_quantize_colwise(const void* x, fos_dtype dt, int64_t rows, int64_t cols,
                                        const fos_config* cfg, float* amax, uint8_t* codes_t,
                                        uint8_t* scales_t, uint8_t* codes, uint8_t* scales,
                                        fos_stream_t stream);

/*
 * fos_swizzle_scales -- the 1x16 block scales of a [rows, cols] tensor
 * (scales [rows, cols/16], as fos_quantize writes them) rearranged into the
 * tiled layout that block-scaled FP4 GEMMs read: the scale matrix is padded
 * with zero bytes to a multiple of 128 rows and 4 columns and cut into
 * 128 x 4 tiles of 512 bytes, stored tile-row by tile-row; inside a tile,
 * scale (32 i + j, k) (i < 4, j < 32, k < 4) is byte 16 j + 4 i + k.
 * out holds fos_swizzled_scales_bytes(rows, cols) bytes (4-byte aligned).
 * The pages pass plain scales to their GEMMs; this is the layout a GEMM
 * library's NVFP4 path takes, checked in the tests against such a GEMM.
 * fos_swizzled_scales_bytes returns -1 for negative sizes or cols % 16 != 0.
 * Errors: FOS_ERR_INVALID_ARG (negative sizes, null or non-device pointers
 * with a nonzero size), FOS_ERR_UNSUPPORTED (cols % 16 != 0),
 * FOS_ERR_MISALIGNED (out not 4-byte aligned).
 */
FOS_API int64_t fos_swizzled_scales_bytes(int64_t rows, int64_t cols);
FOS_API fos_status fos_swizzle_scales(const uint8_t* scales, int64_t rows, int64_t cols,
                                      uint8_t* out, fos_stream_t stream);

/*
 * fos_mm -- out = a . b^T from quantized operands, the forward product of
 * the grouped PR's four_over_six_mm: a [M, K] and b [N, K] were quantized
 * with 1x16 blocks (codes [M, K/2] and [N, K/2]) and their block scales put
 * into the tiled GEMM layout (fos_swizzle_scales, or written there directly
 * by the quantize call with scale_layout = FOS_SCALES_TILED); a_amax /
 * b_amax are the amaxes they were quantized with (a: [M] when
 * cfg->granularity is FOS_SCALE_ROW, else [1]; b: [1]).  One persistent
 * launch of this library's kernel on the tensor cores (tcgen05 block-scaled
 * E2M1 MMAs with UE4M3 scales, fp32 accumulation in tensor memory, one CTA
 * per SM walking 128 x 192 output tiles) forms the block-scaled product D
 * of each tile, and its epilogue applies the global decode scales before
 * the single store,
 *   out[m][n] = (D[m][n] * g_a(m)) * g_b,  g = rn(1 / S),
 * S the global scale fos_quantize used (cfg->e4m3_bound).  out: fp32
 * [M, N] row-major, 16-byte aligned, like all operands.  M and N multiples
 * of 16, K a multiple of 64.  The kernel's waits are bounded: a CTA whose
 * wait gave up (which takes about a second) writes NaN into the first
 * element of its first tile.  Nothing is allocated.
 */
FOS_API fos_status fos_mm(const uint8_t* a_codes, const uint8_t* a_scales_tiled,
                          const float* a_amax, const uint8_t* b_codes,
                          const uint8_t* b_scales_tiled, const float* b_amax, int64_t M,
                          int64_t N, int64_t K, const fos_config* cfg, float* out,
                          fos_stream_t stream);

/*
 * fos_dequantize -- standard NVFP4 decode (grouped PR, first commit:
 * "nvfp4_dequantize: the standard NVFP4 decode (recipe-agnostic)"):
 *   out = round_to(out_dt, e2m1(code) * (e4m3(scale) / S)),
 * with S recomputed from amax and cfg->e4m3_bound exactly as fos_quantize
 * does; the candidate choice need not be stored.  cfg->block and
 * cfg->granularity select the scale layout and the amax indexing;
 * mode / metric / precision are ignored.  out is [rows, cols] of out_dt.
 */
FOS_API fos_status fos_dequantize(const uint8_t* codes, const uint8_t* scales, const float* amax,
                          int64_t rows, int64_t cols, const fos_config* cfg, void* out,
                          fos_dtype out_dt, fos_stream_t stream);

/*
 * fos_qdq -- fused fake-QAT quantize-dequantize of a list of n discrete
 * rank-2 tensors (Megatron PR: "General list API" and "Fused data path":
 * codes and E4M3 scales stay in registers; only the dequantized BF16/FP16
 * result is written).  The whole list is processed in one kernel launch
 * (lists longer than FOS_QDQ_MAX_LIST are split into several launches).
 *   x[i], out[i]: device pointers, rows[i] x cols[i], dtype dt (bf16 or
 *   fp16; out has the same dtype).  amax[i]: device pointer to one float,
 *   the per-tensor amax: read when cfg->amax_is_input, else computed and
 *   written first.  Only 1x16 blocks and FOS_SCALE_TENSOR (the pages'
 *   non-goals exclude 2D blocks and row scaling for this path).
 * The host arrays x, out, rows, cols, amax must hold n entries each; the
 * data pointers of an empty tensor (rows or cols 0) may be null.
 * Result equals fos_dequantize(fos_quantize(x)) bit for bit.
 * Errors: FOS_ERR_INVALID_ARG (n < 0, null arrays or pointers, bad enum,
 * tensors on different devices), FOS_ERR_UNSUPPORTED (fp32, 16x16 blocks,
 * per-row scale, cols % 16 != 0), FOS_ERR_MISALIGNED (x or out not 32-byte
 * aligned).
 */
#define FOS_QDQ_MAX_LIST 64
FOS_API fos_status fos_qdq(int n, const void* const* x, void* const* out, const int64_t* rows,
                   const int64_t* cols, float* const* amax, fos_dtype dt,
                   const fos_config* cfg, fos_stream_t stream);

/*
 * fos_qdq_fused -- fos_qdq with the per-tensor amax computed, in ONE
 * persistent launch (the only other work on the stream is a clear of the
 * workspace): the launch runs the amax pass of tensor 0, then
 * quantize-dequantizes tensor i while it computes the amax of tensor i+1
 * (the Megatron PR, "Fused data path", computes each weight's amax with a
 * separate PyTorch reduction first and lists the per-weight launches among
 * its pending work).  Knobs, layouts and results are those of fos_qdq with
 * cfg->amax_is_input = 0, which this call requires; amax[i] receives tensor
 * i's amax.  n <= FOS_QDQ_MAX_LIST.
 *   workspace: the warps of the launch wait for one another (a tensor's QDQ
 *   starts once its amax is complete) and keep their counters here: device
 *   memory owned by the caller, on the tensors' device, 256-byte aligned, at
 *   least fos_qdq_fused_workspace_bytes(n) bytes.  The call clears it on
 *   `stream` before the launch; calls that may run at the same time need
 *   different workspaces.
 * The launch is cooperative (all of its CTAs resident at once); it returns
 * FOS_ERR_CUDA if the device cannot place them.  Every wait is bounded: one
 * that does not complete within about a second ends the launch with the
 * outputs incomplete and a nonzero code in the workspace, which
 * fos_workspace_error reads.
 */
FOS_API size_t fos_qdq_fused_workspace_bytes(int n);
FOS_API fos_status fos_qdq_fused(int n, const void* const* x, void* const* out,
                                 const int64_t* rows, const int64_t* cols, float* const* amax,
                                 fos_dtype dt, const fos_config* cfg, void* workspace,
                                 size_t workspace_bytes, fos_stream_t stream);

/*
 * fos_qdq_fused_static -- fos_qdq_fused without a workspace argument, for
 * callers that have no way to obtain device memory at the point of the call:
 * code that runs inside another framework's allocator and may not go around
 * it, or a runtime that forbids allocations after its start-up.  The pages
 * have no counterpart; this is a convenience of this library.
 * The counters live in one fixed array of the library (768 bytes on every
 * GPU that loads it, kept until the process exits), so lists are limited to
 * n <= FOS_QDQ_MAX_LIST (64); longer lists return FOS_ERR_UNSUPPORTED.
 * Nothing is allocated: no cudaMalloc, no cudaFree, no allocating library
 * call.  Each call looks up the array's device address on the data's device
 * (with that device current), so a reset of that device's primary context
 * between calls is harmless; while `stream` is being captured the address
 * of the previous lookup is reused instead, so make the first call on a
 * device before any stream capture.  Host-side argument checks are those of
 * fos_qdq_fused, in the same order, and come before any CUDA call.  Each
 * call clears the array on `stream` before its launch.
 * Every call on a device shares the one array: calls whose work may overlap
 * on the GPU (other streams, other threads) race and give wrong results;
 * order them on one stream.  A wait that runs out is recorded in the array
 * (not readable through this call); use fos_qdq_fused with a workspace of
 * your own when that must be checked.  Arguments, results and errors are
 * otherwise those of fos_qdq_fused.
 */
FOS_API fos_status fos_qdq_fused_static(int n, const void* const* x, void* const* out,
                                        const int64_t* rows, const int64_t* cols,
                                        float* const* amax, fos_dtype dt,
                                        const fos_config* cfg, fos_stream_t stream);

/*
 * fos_workspace_error -- waits for `stream` to finish, then stores in *code
 * the error word of a workspace used by fos_qdq_fused: 0 when no wait ran
 * out, 1 when one did.  The one call of this library that synchronises the
 * host (a diagnostic).
 */
FOS_API fos_status fos_workspace_error(const void* workspace, fos_stream_t stream, int* code);

/*
 * fos_quantize_grouped -- one call over a packed MoE token tensor (grouped
 * PR, third commit: "each token group's amax expands to a per-row vector so
 * the whole packed tensor quantizes in one call, bitwise identical to
 * quantizing each group separately"; expert weights flatten to one call).
 *   offs: device int32 [G], cumulative group ends.  Group g covers rows
 *   [end_{g-1}, end_g) with end_{-1} = 0 and end_g = clamp(offs[g],
 *   end_{g-1}, rows).  Rows at or past end_{G-1} (the over-allocated tail of
 *   a padded token dispatcher) are not read; their codes and scales are 0.
 *   With 16x16 blocks offs entries should be multiples of 16; a tile belongs
 *   to the group of its first row.
 *   group_amax: device float [G]; read when cfg->amax_is_input, otherwise
 *   computed (NaN-dropping, empty group -> 0) and written.
 *   cfg->granularity is ignored (the group amax is the global scale source).
 *   1 <= G <= FOS_GROUPED_MAX_GROUPS.
 * Errors: FOS_ERR_INVALID_ARG (G < 1, null pointers, bad enum, pointers on
 * different devices), FOS_ERR_UNSUPPORTED (G above the maximum, cols % 16,
 * 16x16 with rows % 16, a bad bound, the sequential order with 16x16),
 * FOS_ERR_MISALIGNED (x not 32-byte, codes not 8-byte, offs not 4-byte
 * aligned).
 */
#define FOS_GROUPED_MAX_GROUPS 8192
FOS_API fos_status fos_quantize_grouped(const void* x, fos_dtype dt, int64_t rows, int64_t cols,
                                const int32_t* offs, int G, const fos_config* cfg,
                                float* group_amax, uint8_t* codes, uint8_t* scales,
                                fos_stream_t stream);

/*
 * ------------------------------------------------------------------------
 * The feed-forward block around the quantized products: the norm before
 * them, products with an epilogue, and the backward pass of both.
 *
 * 8-bit block format: a tensor [rows, cols], cols % 32 == 0, is held as E4M3
 * codes [rows, cols] (one byte an element) and one UE8M0 scale byte per 32
 * consecutive elements of a row: value = e4m3(code) * 2^(scale - 127).  The
 * scale of a block with largest magnitude a (NaN dropped) is the smallest
 * power of two 2^e, e >= -127, with a <= 448 * 2^e; a code is
 * E4M3_rn_satfinite(v * 2^-e); a NaN element keeps a NaN code.  Scales are
 * plain [rows, cols/32] (FOS_SCALES_PLAIN) or in the tiled layout of
 * fos_swizzle_scales applied to that matrix (FOS_SCALES_TILED, padding
 * zeroed by the call, what the products read): fos_scales8_bytes gives their
 * size, -1 for negative sizes, sizes above 2^30, cols % 32 != 0 or a bad
 * layout.  The workspace sizes below are 0 where a call needs none, and for
 * sizes that it refuses.
 *
 * Sums, the norm's statistics and every step before the one rounding to the
 * output's type are fp32.  Sums have a fixed order: equal calls give equal
 * bits.  Outputs must not overlap inputs or one another, except that an output
 * may be the very tensor of an input where its call says "in the place of".
 * rows and cols below 2^30.  Tensors 32-byte, codes 16-byte (codes_t
 * 32-byte), tiled scales 4-byte, workspaces 256-byte aligned.  Errors:
 * FOS_ERR_INVALID_ARG (bad enum, negative size, missing pointer, codes
 * without scales, pointers on different devices, a workspace too small, an
 * overlap), FOS_ERR_UNSUPPORTED (cols % 32, sizes above the limits),
 * FOS_ERR_MISALIGNED.
 */
FOS_API int64_t fos_scales8_bytes(int64_t rows, int64_t cols, int scale_layout);

/*
 * fos_rms_norm -- h = x + residual (residual may be NULL: h = x), rstd =
 * 1 / sqrt(mean(h^2) + eps) per row, y = h * rstd * weight.  Writes whichever
 * of these is given: h and y rounded to dt, the 8-bit codes and scales of
 * the unrounded y, rstd [rows] fp32 (what the backward pass reads).  weight
 * [cols] is fp32 or of type dt.  eps finite and >= 0.  A row with an infinity
 * has rstd 0; a NaN spreads over its row.  cols == 0 is refused.  h may be in
 * the place of x or of residual.
 */
FOS_API fos_status fos_rms_norm(const void* x, const void* residual, const void* weight,
                                fos_dtype dt, fos_dtype weight_dt, int64_t rows, int64_t cols,
                                float eps, int scale_layout, void* h, void* y, uint8_t* codes,
                                uint8_t* scales, float* rstd, fos_stream_t stream);

/*
 * fos_rms_norm_backward -- with g = dy * weight:
 *   dx = rstd * (g - h * (rstd * mean(g * h * rstd))) + dh
 *   dweight[c] = sum over rows of dy * h * rstd            (fp32)
 * dy, h, dx are of type dt; dh (the gradient that reaches h past the norm)
 * may be NULL; dx is the gradient of x and, the same, of the residual; it may be
 * in the place of dy, h or dh.
 * dweight may be NULL.  With dweight, workspace holds
 * fos_rms_norm_backward_workspace_bytes(rows, cols) bytes of device memory.
 */
FOS_API size_t fos_rms_norm_backward_workspace_bytes(int64_t rows, int64_t cols);
FOS_API fos_status fos_rms_norm_backward(const void* dy, const void* h, const void* dh,
                                         const float* rstd, const void* weight, fos_dtype dt,
                                         fos_dtype weight_dt, int64_t rows, int64_t cols, void* dx,
                                         float* dweight, void* workspace, size_t workspace_bytes,
                                         fos_stream_t stream);

/*
 * fos_quantize8 -- x [rows, cols] in the 8-bit block format along its rows
 * (codes, scales) and / or along its columns: codes_t [cols, R], scales_t of
 * a [cols, R] tensor, R = rows rounded up to a multiple of 32, are the format
 * of x^T with zeros past the last row (the operand of a weight-gradient
 * product, or a weight for the input gradient), from the same read.  Either
 * pair may be NULL.
 */
FOS_API fos_status fos_quantize8(const void* x, fos_dtype dt, int64_t rows, int64_t cols,
                                 int scale_layout, uint8_t* codes, uint8_t* scales,
                                 uint8_t* codes_t, uint8_t* scales_t, fos_stream_t stream);

/* Activations of the product's epilogue: v; max(v, 0); v (1 + erf(v / sqrt 2)) / 2;
 * v (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))) / 2; v / (1 + exp(-v)). */
enum { FOS_ACT_NONE = 0, FOS_ACT_RELU = 1, FOS_ACT_GELU = 2, FOS_ACT_GELU_TANH = 3,
       FOS_ACT_SILU = 4 };

/*
 * fos_act_backward -- d = dout * act'(pre), the gradient at the epilogue's
 * pre-activation (pre as fos_linear8 / fos_linear4 store it; with
 * FOS_ACT_NONE it is not read), in any of: d rounded to dt, its 8-bit rows
 * (for the input gradient's product), its 8-bit columns (for the weight
 * gradient's), and dbias [cols] fp32, the sum of its columns.  dbias over
 * more than 128 rows needs fos_act_backward_workspace_bytes(rows, cols)
 * bytes of workspace.  relu'(0) = 0.  Every finite pre has its derivative (0 or 1
 * far out); an infinite or NaN pre gives NaN, with relu 1, 0 and 0.  d may be in
 * the place of dout or of pre.
 */
FOS_API size_t fos_act_backward_workspace_bytes(int64_t rows, int64_t cols);
FOS_API fos_status fos_act_backward(const void* dout, const void* pre, fos_dtype dt, int64_t rows,
                                    int64_t cols, int act, int scale_layout, void* d,
                                    uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                                    uint8_t* scales_t, float* dbias, void* workspace,
                                    size_t workspace_bytes, fos_stream_t stream);

/* What a product's epilogue does, in this order, in fp32 with one rounding per
 * stored tensor: v = product + bias; pre = v; out = act(v) + residual. */
typedef struct {
    int act;              /* FOS_ACT_*                                          */
    int out_dt;           /* fos_dtype of out, residual and pre                 */
    int bias_dt;          /* fos_dtype of bias: FOS_FP32 or out_dt              */
    const void* bias;     /* [N] or NULL                                        */
    const void* residual; /* [M, N] or NULL                                     */
    void* pre;            /* [M, N] or NULL: kept for fos_act_backward          */
} fos_epilogue;

/*
 * fos_linear8 -- out [M, N] = act(a . b^T + bias) + residual from operands in
 * the 8-bit block format: a [M, K] (tokens) and b [N, K] (weights), codes
 * [M, K] and [N, K], scales tiled.  N % 16 == 0, K % 32 == 0, K > 0; M any
 * number from 0, one token included.  out may be in the place of the residual.
 * fos_linear4 -- the same from NVFP4 operands as fos_mm takes them (1x16
 * codes [M, K/2] and [N, K/2], tiled scales, amaxes; cfg->granularity
 * FOS_SCALE_ROW: a_amax [M]); the product is (D * g_a(m)) * g_b as in fos_mm.
 * Products run on the tensor cores with fp32 accumulation; the order of the
 * sum over K is fixed by the sizes.  out, residual, pre, bias, codes and
 * scales 16-byte aligned.  Waits are bounded as in fos_mm: a CTA whose wait
 * gave up writes NaN into the first element of its first tile.
 */
FOS_API fos_status fos_linear8(const uint8_t* a_codes, const uint8_t* a_scales_tiled,
                               const uint8_t* b_codes, const uint8_t* b_scales_tiled, int64_t M,
                               int64_t N, int64_t K, const fos_epilogue* epilogue, void* out,
                               fos_stream_t stream);
FOS_API fos_status fos_linear4(const uint8_t* a_codes, const uint8_t* a_scales_tiled,
                               const float* a_amax, const uint8_t* b_codes,
                               const uint8_t* b_scales_tiled, const float* b_amax, int64_t M,
                               int64_t N, int64_t K, const fos_config* cfg,
                               const fos_epilogue* epilogue, void* out, fos_stream_t stream);

/*
 * ------------------------------------------------------------------------
 * The experts' part of a feed-forward block.  Rows (tokens) are packed by
 * expert: offs (device int32 [G]) holds the cumulative ends, read as
 * fos_quantize_grouped reads them: expert e has rows [end_{e-1}, end_e),
 * end_e = clamp(offs[e], end_{e-1}, rows).  Any expert may be empty.  The ends
 * are read on the device, so one captured graph serves every routing.  What rows
 * at or past the last end hold does not matter, and what an output holds for them
 * is left as it was.  1 <= G <= FOS_LINEAR_MAX_GROUPS.  Conventions, formats and errors
 * are those of the feed-forward operators above; sizes, and products of two of
 * them, as there (rows x N, G x N x K and so on up to 2^40, G x N below 2^31).
 */
#define FOS_LINEAR_MAX_GROUPS 1024

/*
 * fos_linear8_grouped, fos_linear4_grouped -- fos_linear8 / fos_linear4 with the
 * weights of each row's expert:
 *   out[m] = act(a[m] . b[e]^T + bias[e]) + residual[m],  e the expert of row m.
 *   a_codes [rows, K] ([rows, K/2]) with PLAIN scales [rows, K/32] ([rows, K/16]):
 *     what fos_rms_norm, fos_quantize8, fos_act_backward with FOS_SCALES_PLAIN
 *     (fos_quantize_grouped, fos_quantize) write for the packed rows;
 *   b_codes [G, N, K] ([G, N, K/2]), b_scales_tiled: each expert's tiled scales,
 *     one after the other (with N % 128 == 0 that is one quantize call's output for
 *     the weights [G * N, K]);
 *   a_amax [G] (FOS_SCALE_TENSOR: what fos_quantize_grouped returns) or [rows]
 *     (FOS_SCALE_ROW); b_amax [G].
 *   epilogue: bias [G, N]; residual, pre and out [rows, N].
 * N % 16 == 0; K a multiple of 128 (64).  With the weights' column-wise form as b
 * the 8-bit call is also the input gradient.  Waits are bounded as in fos_linear8.
 */
FOS_API fos_status fos_linear8_grouped(const uint8_t* a_codes, const uint8_t* a_scales,
                                       const uint8_t* b_codes, const uint8_t* b_scales_tiled,
                                       const int32_t* offs, int G, int64_t rows, int64_t N,
                                       int64_t K, const fos_epilogue* epilogue, void* out,
                                       fos_stream_t stream);
FOS_API fos_status fos_linear4_grouped(const uint8_t* a_codes, const uint8_t* a_scales,
                                       const float* a_amax, const uint8_t* b_codes,
                                       const uint8_t* b_scales_tiled, const float* b_amax,
                                       const int32_t* offs, int G, int64_t rows, int64_t N,
                                       int64_t K, const fos_config* cfg,
                                       const fos_epilogue* epilogue, void* out,
                                       fos_stream_t stream);

/*
 * fos_quantize8_grouped, fos_act_backward_grouped -- fos_quantize8 / fos_act_backward
 * of packed rows.  codes, scales (plain) and d are as there.  The column-wise form
 * has P = fos_grouped_cols(rows, G) columns: expert e's rows are columns p_e ...,
 * p_0 = 0, p_{e+1} = p_e + 128 ceil(n_e / 128), with zeros up to p_{e+1}, so that each
 * expert's part is an operand by itself; codes_t [cols, P], scales_t the tiled scales
 * of a [cols, P] tensor.  What they hold past the last expert's part is left as it
 * was (but the padding of scales_t's rows to 128, zeros everywhere).  dbias [G, cols] fp32: the sum of each expert's rows (0 for an empty one); it
 * needs fos_act_backward_grouped_workspace_bytes(rows, cols, G) bytes of workspace.
 * fos_grouped_cols returns -1 for negative rows or a G out of range.
 */
FOS_API int64_t fos_grouped_cols(int64_t rows, int G);
FOS_API fos_status fos_quantize8_grouped(const void* x, fos_dtype dt, int64_t rows, int64_t cols,
                                         const int32_t* offs, int G, uint8_t* codes,
                                         uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t,
                                         fos_stream_t stream);
FOS_API size_t fos_act_backward_grouped_workspace_bytes(int64_t rows, int64_t cols, int G);
FOS_API fos_status fos_act_backward_grouped(const void* dout, const void* pre, fos_dtype dt,
                                            int64_t rows, int64_t cols, const int32_t* offs, int G,
                                            int act, void* d, uint8_t* codes, uint8_t* scales,
                                            uint8_t* codes_t, uint8_t* scales_t, float* dbias,
                                            void* workspace, size_t workspace_bytes,
                                            fos_stream_t stream);

/*
 * fos_linear8_grouped_wgrad -- the experts' weight gradients,
 *   out[e] = d_t[:, e] . z_t[:, e]^T + residual[e]          [G, N, K]
 * from the column-wise forms of the gradient behind the product (d_codes_t [N, P],
 * d_scales_t tiled) and of its input (z_codes_t [K, P], z_scales_t tiled) for the same
 * offs, P = fos_grouped_cols(rows, G).  An expert without rows gets its residual, or
 * zeros.  out and residual (may be NULL; out may be in its place) are of out_dt, 16-byte
 * aligned.  N % 16 == 0, K % 16 == 0, K > 0.
 */
FOS_API fos_status fos_linear8_grouped_wgrad(const uint8_t* d_codes_t, const uint8_t* d_scales_t,
                                             const uint8_t* z_codes_t, const uint8_t* z_scales_t,
                                             const int32_t* offs, int G, int64_t rows, int64_t N,
                                             int64_t K, const void* residual, fos_dtype out_dt,
                                             void* out, fos_stream_t stream);

/*
 * fos_matvec4 -- few rows of x, not quantized, with NVFP4 weights:
 *   out[p] = act(x[p / (M / x_rows)] . b[e]^T + bias[e]) + residual[p],  e = ids[p]
 * x [x_rows, K] of dt; ids (device int32 [M]) or NULL (e = 0, G = 1); x_rows divides M:
 * the experts of one token stand next to one another, or every row has its own x.
 * b_codes [G, N, K/2], b_scales_tiled and b_amax [G] as in fos_linear4_grouped;
 * cfg->granularity is not read.  epilogue bias [G, N]; residual and out [M, N] (out may be
 * in the residual's place); pre must be NULL.  A row whose id is outside 0 .. G - 1 is
 * left as it was.  Weights are decoded exactly, x is taken as it is (no element is rounded,
 * whatever stands beside it) and products are summed in fp32.  An expert's weights are
 * read again for every eight rows (two of fp32 x): for a few rows; from 16 on (4 of fp32)
 * fos_linear4 of quantized rows takes less.  Rows with elements below 2^-31 (fp32: 2^-37)
 * of the largest of their 128 neighbours take longer.  M <= FOS_MATVEC_MAX_ROWS;
 * G <= FOS_LINEAR_MAX_GROUPS; N % 16 == 0; K % 32 == 0, K > 0.  x, codes, scales and the
 * epilogue's tensors 16-byte aligned.
 */
#define FOS_MATVEC_MAX_ROWS 1024
FOS_API fos_status fos_matvec4(const void* x, fos_dtype dt, int64_t x_rows, const int32_t* ids,
                               const uint8_t* b_codes, const uint8_t* b_scales_tiled,
                               const float* b_amax, int64_t M, int64_t N, int64_t K, int G,
                               const fos_config* cfg, const fos_epilogue* epilogue, void* out,
                               fos_stream_t stream);

/* Static, human-readable name of a status code. */
FOS_API const char* fos_status_string(fos_status s);

/* Library version as major * 10000 + minor * 100 + patch. */
FOS_API int fos_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FOS_H */
