"""NVFP4 four-over-six block quantizer for GB300 -- Python binding.

Argument marshalling only: every step of the quantizer runs in the CUDA
kernels of ``libfos.so`` (C ABI in ``include/fos.h``).  PyTorch supplies the
device memory and the current stream.  There is no CPU path: if the library
is not built, or a tensor is not on a CUDA device, the call raises.

Entry points (names follow the C ABI):
  amax(x, granularity)                      -> float32 amax
  quantize(x, ...)                          -> (codes, scales, amax)
  check_tile_amax(amax)                     -> number of non-uniform 16-row tiles
  quantize_list(xs, ...)                    -> ([codes], [scales], [amax])
  quantize_overlap(x, amax, codes, scales, x_next, amax_next)
  dequantize(codes, scales, amax, ...)      -> tensor
  qdq(xs, ...)                              -> list of tensors (one launch)
  qdq_fused(xs, ...)                        -> (outs, amaxes), every amax in the same launch
  workspace_error(workspace)                -> error word of a fused launch
  quantize_grouped(x, offs, ...)            -> (codes, scales, group_amax)
  quantize_colwise(x, ...)                  -> (codes_t, scales_t, amax[, codes, scales])
  swizzle_scales(scales, rows, cols)        -> scales in the tiled GEMM layout
  mm(a_codes, a_tiled, a_amax, b_codes, b_tiled, b_amax) -> fp32 a . b^T
  rms_norm(x, weight, residual, ...)        -> (codes, scales, y, h, rstd), 8-bit blocks
  rms_norm_backward(dy, h, rstd, weight, dh) -> (dx, dweight)
  quantize8(x, ...)                         -> (codes, scales, codes_t, scales_t)
  linear8(a_codes, a_scales, b_codes, b_scales, ...) -> act(a . b^T + bias) + residual
  linear4(a_codes, a_scales, a_amax, b_codes, b_scales, b_amax, ...) -> the same, NVFP4
  act_backward(dout, pre, act, ...)         -> (codes, scales, codes_t, scales_t, d, dbias)
  linear8_grouped(a_codes, a_scales, b_codes, b_scales, offs, ...) -> linear8 of rows packed by expert
  linear4_grouped(a_codes, a_scales, a_amax, b_codes, b_scales, b_amax, offs, ...) -> the same, NVFP4
  quantize8_grouped(x, offs, ...)           -> (codes, scales, codes_t, scales_t), columns by expert
  act_backward_grouped(dout, pre, act, offs, ...) -> act_backward likewise, dbias [G, cols]
  linear8_grouped_wgrad(d_codes_t, d_scales_t, z_codes_t, z_scales_t, offs, rows) -> [G, N, K]
  matvec4(x, b_codes, b_scales, b_amax, ids, ...) -> few unquantized rows times NVFP4 weights
  release_workspaces()                      -> what the backward calls keep for this thread
"""
import ctypes
import os
import threading
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfos.so")

(FOS_OK, FOS_ERR_INVALID_ARG, FOS_ERR_UNSUPPORTED, FOS_ERR_MISALIGNED, FOS_ERR_CUDA,
 FOS_ERR_NONUNIFORM_TILE_AMAX) = range(6)
FOS_BF16, FOS_FP16, FOS_FP32 = 0, 1, 2
QDQ_MAX_LIST = 64
GROUPED_MAX_GROUPS = 8192
LINEAR_MAX_GROUPS = 1024
MATVEC_MAX_ROWS = 1024

_DT = {torch.bfloat16: FOS_BF16, torch.float16: FOS_FP16, torch.float32: FOS_FP32}
_NAMES = ("fos_amax", "fos_quantize", "fos_quantize_list", "fos_quantize_overlap",
          "fos_dequantize", "fos_qdq", "fos_quantize_grouped",
          "fos_status_string", "fos_version", "fos_diag_convert")


class FosError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (what, status_string(status), status))


class FosConfig(ctypes.Structure):
    _fields_ = [("block", ctypes.c_int), ("mode", ctypes.c_int), ("err_metric", ctypes.c_int),
                ("err_precision", ctypes.c_int), ("e4m3_bound", ctypes.c_int),
                ("granularity", ctypes.c_int), ("amax_is_input", ctypes.c_int),
                ("err_order", ctypes.c_int), ("scale_layout", ctypes.c_int)]


class FosEpilogue(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int), ("out_dt", ctypes.c_int), ("bias_dt", ctypes.c_int),
                ("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("pre", ctypes.c_void_p)]


@dataclass(frozen=True)
class Config:
    """Knobs of the quantizer (see include/fos.h)."""
    block16x16: bool = False
    four_over_six: bool = True
    mse: bool = True
    err_f16: bool = False
    bound: int = 448
    row_scaled: bool = False
    seq_order: bool = False  # sum a block's error terms in element order (1x16 only)
    scale_tiled: bool = False  # write scales in the tiled GEMM layout (1x16 only)

    def c(self, amax_is_input):
        return FosConfig(int(self.block16x16), int(self.four_over_six), int(self.mse),
                         int(self.err_f16), int(self.bound), int(self.row_scaled),
                         int(bool(amax_is_input)), int(self.seq_order),
                         int(self.scale_tiled))


_lib = None


def lib():
    """The loaded libfos.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libfos.so is not built (run __graft_entry__.build() or "
                               "python -m nvfp4_quantization_precision_gb300.build)")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        CFG = ctypes.POINTER(FosConfig)
        L.fos_amax.argtypes = [P, I, I64, I64, I, P, P]
        L.fos_quantize.argtypes = [P, I, I64, I64, CFG, P, P, P, P]
        L.fos_quantize_list.argtypes = [I, P, I, P, P, CFG, P, P, P, P]
        L.fos_quantize_overlap.argtypes = [P, I, I64, I64, CFG, P, P, P, P, I64, I64, P, P]
        L.fos_dequantize.argtypes = [P, P, P, I64, I64, CFG, P, I, P]
        L.fos_qdq.argtypes = [I, P, P, P, P, P, I, CFG, P]
        L.fos_quantize_grouped.argtypes = [P, I, I64, I64, P, I, CFG, P, P, P, P]
        L.fos_diag_convert.argtypes = [I, P, P, I64, P]
        L.fos_qdq_fused_workspace_bytes.argtypes = [I]
        L.fos_qdq_fused_workspace_bytes.restype = ctypes.c_size_t
        L.fos_qdq_fused.argtypes = [I, P, P, P, P, P, I, CFG, P, ctypes.c_size_t, P]
        L.fos_workspace_error.argtypes = [P, P, ctypes.POINTER(I)]
        L.fos_check_tile_amax.argtypes = [P, I64, P, P]
        L.fos_tile_amax_status.argtypes = [P, P]
        L.fos_swizzled_scales_bytes.argtypes = [I64, I64]
        L.fos_swizzled_scales_bytes.restype = ctypes.c_int64
        for n in ("fos_check_tile_amax", "fos_tile_amax_status", "fos_amax", "fos_quantize", "fos_quantize_list", "fos_quantize_overlap",
                  "fos_dequantize", "fos_qdq", "fos_qdq_fused", "fos_workspace_error",
                  "fos_quantize_grouped", "fos_diag_convert"):
            getattr(L, n).restype = ctypes.c_int
        L.fos_scales8_bytes.argtypes = [I64, I64, I]
        L.fos_scales8_bytes.restype = ctypes.c_int64
        L.fos_rms_norm.argtypes = [P, P, P, I, I, I64, I64, ctypes.c_float, I, P, P, P, P, P, P]
        L.fos_rms_norm_backward.argtypes = [P, P, P, P, P, I, I, I64, I64, P, P, P,
                                            ctypes.c_size_t, P]
        L.fos_quantize8.argtypes = [P, I, I64, I64, I, P, P, P, P, P]
        L.fos_act_backward.argtypes = [P, P, I, I64, I64, I, I, P, P, P, P, P, P, P,
                                       ctypes.c_size_t, P]
        EP = ctypes.POINTER(FosEpilogue)
        L.fos_linear8.argtypes = [P, P, P, P, I64, I64, I64, EP, P, P]
        L.fos_linear4.argtypes = [P, P, P, P, P, P, I64, I64, I64, CFG, EP, P, P]
        for n in ("fos_rms_norm", "fos_rms_norm_backward", "fos_quantize8", "fos_act_backward",
                  "fos_linear8", "fos_linear4"):
            getattr(L, n).restype = ctypes.c_int
        for n in ("fos_rms_norm_backward_workspace_bytes", "fos_act_backward_workspace_bytes"):
            getattr(L, n).argtypes = [I64, I64]
            getattr(L, n).restype = ctypes.c_size_t
        L.fos_linear8_grouped.argtypes = [P, P, P, P, P, I, I64, I64, I64, EP, P, P]
        L.fos_linear4_grouped.argtypes = [P, P, P, P, P, P, P, I, I64, I64, I64, CFG, EP, P, P]
        L.fos_quantize8_grouped.argtypes = [P, I, I64, I64, P, I, P, P, P, P, P]
        L.fos_act_backward_grouped.argtypes = [P, P, I, I64, I64, P, I, I, P, P, P, P, P, P, P,
                                               ctypes.c_size_t, P]
        L.fos_linear8_grouped_wgrad.argtypes = [P, P, P, P, P, I, I64, I64, I64, P, I, P, P]
        L.fos_matvec4.argtypes = [P, I, I64, P, P, P, P, I64, I64, I64, I, CFG, EP, P, P]
        for n in ("fos_linear8_grouped", "fos_linear4_grouped", "fos_quantize8_grouped",
                  "fos_act_backward_grouped", "fos_linear8_grouped_wgrad", "fos_matvec4"):
            getattr(L, n).restype = ctypes.c_int
        L.fos_grouped_cols.argtypes = [I64, I]
        L.fos_grouped_cols.restype = ctypes.c_int64
        L.fos_act_backward_grouped_workspace_bytes.argtypes = [I64, I64, I]
        L.fos_act_backward_grouped_workspace_bytes.restype = ctypes.c_size_t
        L.fos_status_string.argtypes = [I]
        L.fos_status_string.restype = ctypes.c_char_p
        L.fos_version.restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(s):
    return lib().fos_status_string(int(s)).decode()


def _check(rc, what):
    if rc != FOS_OK:
        raise FosError(rc, what)


# The current stream's handle without building a torch.cuda.Stream (2.2 us a
# call on the host), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t):
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _cuda(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _p(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def amax(x, row_scaled=False, out=None):
    """NaN-dropping max|x| per tensor ([1]) or per row ([rows]), float32."""
    _cuda(x, "x")
    R, C = x.shape
    n = R if row_scaled else 1
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=x.device)
    _check(lib().fos_amax(_p(x), _DT[x.dtype], R, C, int(row_scaled), _p(out), _stream(x)),
           "fos_amax")
    return out


def scales_shape(rows, cols, block16x16):
    return (rows // 16 if block16x16 else rows, cols // 16)


def _scales_buffer(rows, cols, cfg, dev):
    """The scale output of a quantize of [rows, cols] under cfg: [rows, cols/16]
    (plain), or the flat tiled buffer of fos_swizzled_scales_bytes bytes."""
    if cfg.scale_tiled:
        nbytes = lib().fos_swizzled_scales_bytes(rows, cols)
        if nbytes < 0:
            raise ValueError("bad shape for tiled scales")
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return torch.empty(scales_shape(rows, cols, cfg.block16x16), dtype=torch.uint8, device=dev)


def check_tile_amax(amax, bad=None):
    """Number of 16-row tiles of a per-row amax [rows] whose entries are not
    all bitwise equal (fos_check_tile_amax); reads the count back, so it
    waits for the stream."""
    _cuda(amax, "amax")
    if bad is None:
        bad = torch.empty(1, dtype=torch.int64, device=amax.device)
    _check(lib().fos_check_tile_amax(_p(amax), amax.numel(), _p(bad), _stream(amax)),
           "fos_check_tile_amax")
    return int(bad.item())


def quantize(x, cfg=Config(), amax=None, codes=None, scales=None, amax_given=None,
             validate=False):
    """Quantize x [rows, cols] (bf16 / fp16 / fp32).  amax is read when
    given (the default when a tensor is passed); with amax_given=False it is
    an output buffer the library fills.  With amax=None it is allocated,
    computed and returned.  validate=True checks a given per-row amax of a
    16x16 quantize for tile uniformity first (fos_check_tile_amax and
    fos_tile_amax_status, which wait for the stream) and raises FosError
    with FOS_ERR_NONUNIFORM_TILE_AMAX when a tile's rows differ."""
    _cuda(x, "x")
    R, C = x.shape
    dev = x.device
    given = (amax is not None) if amax_given is None else bool(amax_given)
    if validate and given and cfg.block16x16 and cfg.row_scaled:
        _cuda(amax, "amax")
        bad = torch.empty(1, dtype=torch.int64, device=dev)
        _check(lib().fos_check_tile_amax(_p(amax), amax.numel(), _p(bad), _stream(amax)),
               "fos_check_tile_amax")
        _check(lib().fos_tile_amax_status(_p(bad), _stream(amax)), "fos_quantize")
    if amax is None:
        amax = torch.empty(R if cfg.row_scaled else 1, dtype=torch.float32, device=dev)
    if codes is None:
        codes = torch.empty((R, C // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = _scales_buffer(R, C, cfg, dev)
    cc = cfg.c(given)
    _check(lib().fos_quantize(_p(x), _DT[x.dtype], R, C, ctypes.byref(cc), _p(amax), _p(codes),
                              _p(scales), _stream(x)), "fos_quantize")
    return codes, scales, amax


def quantize_list(xs, cfg=Config(), amaxes=None, codes=None, scales=None, amax_given=None):
    """fos_quantize over a list of tensors of one dtype (see fos_quantize_list:
    with per-tensor scale and amax computed, the amax pass of tensor i+1 runs
    inside the encode launch of tensor i).  Returns (codes, scales, amaxes)
    lists."""
    n = len(xs)
    if n == 0:
        return [], [], []
    for x in xs:
        _cuda(x, "x")
    dt = xs[0].dtype
    given = (amaxes is not None) if amax_given is None else bool(amax_given)
    dev = xs[0].device
    if amaxes is None:
        amaxes = [torch.empty(x.shape[0] if cfg.row_scaled else 1, dtype=torch.float32,
                              device=dev) for x in xs]
    if codes is None:
        codes = [torch.empty((x.shape[0], x.shape[1] // 2), dtype=torch.uint8, device=dev)
                 for x in xs]
    if scales is None:
        scales = [_scales_buffer(x.shape[0], x.shape[1], cfg, dev) for x in xs]
    P = ctypes.c_void_p * n
    xp = P(*[x.data_ptr() for x in xs])
    ap = P(*[a.data_ptr() for a in amaxes])
    cp = P(*[c.data_ptr() for c in codes])
    sp = P(*[s.data_ptr() for s in scales])
    rows = (ctypes.c_int64 * n)(*[x.shape[0] for x in xs])
    cols = (ctypes.c_int64 * n)(*[x.shape[1] for x in xs])
    cc = cfg.c(given)
    _check(lib().fos_quantize_list(n, xp, _DT[dt], rows, cols, ctypes.byref(cc), ap, cp, sp,
                                   _stream(xs[0])), "fos_quantize_list")
    return codes, scales, amaxes


def quantize_overlap(x, amax, codes, scales, x_next=None, amax_next=None, cfg=Config()):
    """Quantize x with its per-tensor amax given (1x16) and compute the amax
    of x_next in the same launch (fos_quantize_overlap)."""
    _cuda(x, "x")
    R, C = x.shape
    if x_next is not None:
        _cuda(x_next, "x_next")
        Rn, Cn = x_next.shape
    else:
        Rn = Cn = 0
    cc = cfg.c(True)
    _check(lib().fos_quantize_overlap(_p(x), _DT[x.dtype], R, C, ctypes.byref(cc), _p(amax),
                                      _p(codes), _p(scales), _p(x_next), Rn, Cn, _p(amax_next),
                                      _stream(x)), "fos_quantize_overlap")
    return codes, scales


def dequantize(codes, scales, amax, cfg=Config(), out_dtype=torch.bfloat16, out=None):
    _cuda(codes, "codes")
    R, C2 = codes.shape
    C = 2 * C2
    if out is None:
        out = torch.empty((R, C), dtype=out_dtype, device=codes.device)
    cc = cfg.c(True)
    _check(lib().fos_dequantize(_p(codes), _p(scales), _p(amax), R, C, ctypes.byref(cc), _p(out),
                                _DT[out.dtype], _stream(codes)), "fos_dequantize")
    return out


def qdq(xs, cfg=Config(), amaxes=None, outs=None, amax_given=None):
    """Fused quantize-dequantize of a list of rank-2 bf16/fp16 tensors in one
    launch.  amaxes: list of 1-element float32 tensors, read when given (the
    default when passed) or filled when amax_given=False; None allocates and
    computes them.  Returns the list of outputs."""
    n = len(xs)
    if n == 0:
        return []
    for x in xs:
        _cuda(x, "x")
    dt = xs[0].dtype
    given = (amaxes is not None) if amax_given is None else bool(amax_given)
    if amaxes is None:
        amaxes = [torch.empty(1, dtype=torch.float32, device=x.device) for x in xs]
    if outs is None:
        outs = [torch.empty_like(x) for x in xs]
    P = ctypes.c_void_p * n
    xp = P(*[x.data_ptr() for x in xs])
    op = P(*[o.data_ptr() for o in outs])
    ap = P(*[a.data_ptr() for a in amaxes])
    rows = (ctypes.c_int64 * n)(*[x.shape[0] for x in xs])
    cols = (ctypes.c_int64 * n)(*[x.shape[1] for x in xs])
    cc = cfg.c(given)
    _check(lib().fos_qdq(n, xp, op, rows, cols, ap, _DT[dt], ctypes.byref(cc), _stream(xs[0])),
           "fos_qdq")
    return outs


def quantize_colwise(x, cfg=Config(), amax=None, codes_t=None, scales_t=None, rowwise=False,
                     codes=None, scales=None, amax_given=None):
    """fos_quantize_colwise: the quantization of x.T from x (1x16, per-tensor
    scale).  With rowwise=True (or codes/scales passed) the row-wise result
    of x comes from the same read.  Returns (codes_t, scales_t, amax) or
    (codes_t, scales_t, amax, codes, scales)."""
    _cuda(x, "x")
    R, C = x.shape
    dev = x.device
    given = (amax is not None) if amax_given is None else bool(amax_given)
    if amax is None:
        amax = torch.empty(1, dtype=torch.float32, device=dev)
    if codes_t is None:
        codes_t = torch.empty((C, R // 2), dtype=torch.uint8, device=dev)
    if scales_t is None:
        scales_t = _scales_buffer(C, R, cfg, dev)
    dual = rowwise or codes is not None or scales is not None
    if dual and codes is None:
        codes = torch.empty((R, C // 2), dtype=torch.uint8, device=dev)
    if dual and scales is None:
        scales = _scales_buffer(R, C, cfg, dev)
    L = lib()
    if not getattr(L, "_colwise_declared", False):
        P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.fos_quantize_colwise.argtypes = [P, I, I64, I64, ctypes.POINTER(FosConfig), P, P, P, P,
                                           P, P]
        L.fos_quantize_colwise.restype = I
        L._colwise_declared = True
    cc = cfg.c(given)
    _check(L.fos_quantize_colwise(_p(x), _DT[x.dtype], R, C, ctypes.byref(cc), _p(amax),
                                  _p(codes_t), _p(scales_t), _p(codes), _p(scales), _stream(x)),
           "fos_quantize_colwise")
    if dual:
        return codes_t, scales_t, amax, codes, scales
    return codes_t, scales_t, amax


def swizzle_scales(scales, rows, cols, out=None):
    """fos_swizzle_scales: 1x16 scales [rows, cols/16] in the tiled layout of
    block-scaled FP4 GEMMs (a flat uint8 tensor, zero padded)."""
    _cuda(scales, "scales")
    L = lib()
    if not getattr(L, "_swizzle_declared", False):
        L.fos_swizzled_scales_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64]
        L.fos_swizzled_scales_bytes.restype = ctypes.c_int64
        L.fos_swizzle_scales.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_void_p, ctypes.c_void_p]
        L.fos_swizzle_scales.restype = ctypes.c_int
        L._swizzle_declared = True
    nbytes = L.fos_swizzled_scales_bytes(rows, cols)
    if nbytes < 0:
        raise ValueError("bad shape for swizzled scales")
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=scales.device)
    _check(L.fos_swizzle_scales(_p(scales), rows, cols, _p(out), _stream(scales)),
           "fos_swizzle_scales")
    return out


def mm(a_codes, a_scales_tiled, a_amax, b_codes, b_scales_tiled, b_amax, cfg=Config(),
       out=None):
    """fos_mm: a . b^T (fp32 [M, N]) from a's and b's 1x16 codes, tiled scales
    (swizzle_scales) and amaxes; cfg.row_scaled when a was quantized with a
    per-row scale."""
    _cuda(a_codes, "a_codes")
    M, K2 = a_codes.shape
    N = b_codes.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=a_codes.device)
    L = lib()
    if not getattr(L, "_mm_declared", False):
        P = ctypes.c_void_p
        L.fos_mm.argtypes = [P, P, P, P, P, P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                             ctypes.POINTER(FosConfig), P, P]
        L.fos_mm.restype = ctypes.c_int
        L._mm_declared = True
    cc = cfg.c(True)
    _check(L.fos_mm(_p(a_codes), _p(a_scales_tiled), _p(a_amax), _p(b_codes), _p(b_scales_tiled),
                    _p(b_amax), M, N, 2 * K2, ctypes.byref(cc), _p(out), _stream(a_codes)),
           "fos_mm")
    return out


def qdq_fused_workspace(n, device):
    """A workspace for fos_qdq_fused over n tensors (caller-side allocation)."""
    nb = lib().fos_qdq_fused_workspace_bytes(int(n))
    return torch.empty(max(nb, 256), dtype=torch.uint8, device=device)


def qdq_fused(xs, cfg=Config(), amaxes=None, outs=None, workspace=None):
    """fos_qdq_fused: amax of every tensor and the fused quantize-dequantize
    of the list in one persistent launch.  amaxes (outputs) and outs are
    allocated when None; workspace too (see qdq_fused_workspace).  Returns
    (outs, amaxes)."""
    n = len(xs)
    if n == 0:
        return [], []
    for x in xs:
        _cuda(x, "x")
    dev = xs[0].device
    if amaxes is None:
        amaxes = [torch.empty(1, dtype=torch.float32, device=dev) for _ in xs]
    if outs is None:
        outs = [torch.empty_like(x) for x in xs]
    if workspace is None:
        workspace = qdq_fused_workspace(n, dev)
    P = ctypes.c_void_p * n
    xp = P(*[x.data_ptr() for x in xs])
    op = P(*[o.data_ptr() for o in outs])
    ap = P(*[a.data_ptr() for a in amaxes])
    rows = (ctypes.c_int64 * n)(*[x.shape[0] for x in xs])
    cols = (ctypes.c_int64 * n)(*[x.shape[1] for x in xs])
    cc = cfg.c(False)
    _check(lib().fos_qdq_fused(n, xp, op, rows, cols, ap, _DT[xs[0].dtype], ctypes.byref(cc),
                               _p(workspace), workspace.numel(), _stream(xs[0])),
           "fos_qdq_fused")
    return outs, amaxes


def workspace_error(workspace):
    """The error word of a fused-launch workspace (waits for the stream)."""
    code = ctypes.c_int(0)
    _check(lib().fos_workspace_error(_p(workspace), _stream(workspace), ctypes.byref(code)),
           "fos_workspace_error")
    return code.value


def quantize_grouped(x, offs, cfg=Config(), group_amax=None, codes=None, scales=None,
                     amax_given=None):
    """One call over a packed token tensor split into groups by cumulative
    ends offs (int32, device).  Rows past offs[-1] get zero codes/scales."""
    _cuda(x, "x")
    _cuda(offs, "offs")
    if offs.dtype != torch.int32:
        raise ValueError("offs must be int32")
    R, C = x.shape
    G = offs.numel()
    dev = x.device
    given = (group_amax is not None) if amax_given is None else bool(amax_given)
    if group_amax is None:
        group_amax = torch.empty(G, dtype=torch.float32, device=dev)
    if codes is None:
        codes = torch.empty((R, C // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty(scales_shape(R, C, cfg.block16x16), dtype=torch.uint8, device=dev)
    cc = cfg.c(given)
    _check(lib().fos_quantize_grouped(_p(x), _DT[x.dtype], R, C, _p(offs), G, ctypes.byref(cc),
                                      _p(group_amax), _p(codes), _p(scales), _stream(x)),
           "fos_quantize_grouped")
    return codes, scales, group_amax


# ------------------------------------------------------------------ feed-forward operators
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = range(5)
_ACTS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH,
         "silu": ACT_SILU}


def _act(act):
    if act not in _ACTS:
        raise ValueError("act must be one of %s" % ", ".join(_ACTS))
    return _ACTS[act]


def _a(t):
    """Address of an optional tensor (None: null)."""
    return t.data_ptr() if t is not None else None


def _like(t, name, shape, dtype, dev):
    """Checks an operand or a caller's output buffer: a contiguous tensor of
    this shape and type on CUDA device number dev."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on cuda:%d"
                         % (name, dtype, tuple(shape), dev))
    return t


def _data(t, name):
    """Checks a rank-2 floating-point input; returns (shape, type, device number)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        _cuda(t, name)
    dt = _DT.get(t.dtype)
    shape = t.shape
    if dt is None or len(shape) != 2:
        raise ValueError("%s must be a rank-2 bf16, fp16 or fp32 tensor" % name)
    return shape, dt, t.get_device()


_DEVICES = [torch.device("cuda", i) for i in range(64)]


def _new(shape, dtype, dev):
    return torch.empty(shape, dtype=dtype, device=_DEVICES[dev])


def _weight(w, cols, dtype, dev):
    wt = w.dtype
    if wt is not torch.float32 and wt is not dtype:
        raise ValueError("weight must be float32 or of the input's type")
    _like(w, "weight", (cols,), wt, dev)
    return _DT[wt]


def _pair8(rows, cols, tiled, codes, scales, dev, names=("codes", "scales")):
    """Code and scale buffers of a [rows, cols] tensor in the 8-bit block
    format: the caller's, checked, or new ones."""
    if cols % 32:
        raise FosError(FOS_ERR_UNSUPPORTED, names[0])
    if codes is None:
        codes = _new((rows, cols), torch.uint8, dev)
    else:
        _like(codes, names[0], (rows, cols), torch.uint8, dev)
    shape = ((rows + 127) // 128 * ((cols + 127) // 128) * 512,) if tiled else (rows, cols // 32)
    if scales is None:
        scales = _new(shape, torch.uint8, dev)
    else:
        _like(scales, names[1], shape, torch.uint8, dev)
    return codes, scales


def scales8_shape(rows, cols, tiled=True):
    """Shape of the scale bytes of a [rows, cols] tensor in the 8-bit block format."""
    n = lib().fos_scales8_bytes(int(rows), int(cols), int(bool(tiled)))
    if n < 0:
        raise ValueError("bad shape for 8-bit block scales")
    return (n,) if tiled else (rows, cols // 32)


def rms_norm(x, weight, residual=None, eps=1e-6, scale_tiled=True, quantized=True,
             normalized=False, codes=None, scales=None, y=None, h=None, rstd=None):
    """fos_rms_norm: h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight
    over the rows of x [rows, cols].  Returns (codes, scales, y, h, rstd):
    y's 8-bit codes and scales (None without quantized), y itself with
    normalized (else None), h (x itself without a residual) and rstd [rows].
    h may be passed as x or as residual, to be written in its place."""
    shape, dt, dev = _data(x, "x")
    R, C = shape
    wdt = _weight(weight, C, x.dtype, dev)
    if residual is not None:
        _like(residual, "residual", shape, x.dtype, dev)
        h = torch.empty_like(x) if h is None else _like(h, "h", shape, x.dtype, dev)
    elif h is not None:
        raise ValueError("h is an output of a norm with a residual")
    if quantized:
        codes, scales = _pair8(R, C, scale_tiled, codes, scales, dev)
    else:
        codes = scales = None
    if normalized:
        y = torch.empty_like(x) if y is None else _like(y, "y", shape, x.dtype, dev)
    else:
        y = None
    if rstd is None:
        rstd = _new((R,), torch.float32, dev)
    else:
        _like(rstd, "rstd", (R,), torch.float32, dev)
    _check(lib().fos_rms_norm(x.data_ptr(), _a(residual), weight.data_ptr(), dt, wdt, R, C, eps,
                              1 if scale_tiled else 0, _a(h), _a(y), _a(codes), _a(scales),
                              rstd.data_ptr(), _stream(x)), "fos_rms_norm")
    return codes, scales, y, x if h is None else h, rstd


# Workspaces of calls that bring none, one per thread, device and stream: two
# threads may interleave the launches of their calls on one stream, and calls on
# different streams overlap.  (An allocation in every call costs 5 to 6 of 16 to
# 27 us on the host.)  Larger ones and those of a captured graph, which may be
# replayed on any stream, are allocated by the call.  A thread keeps those of the
# streams it used last; what it gives up or leaves behind goes back to the
# allocator of the stream that used it, which orders its next use.
_KEPT_MOST = 16 << 20
_KEPT_STREAMS = 8
_kept = threading.local()


def _workspace(workspace, need, dev):
    if need == 0:
        return None, 0
    if workspace is None:
        if need > _KEPT_MOST or _raw_stream is None or torch.cuda.current_device() != dev or \
                torch.cuda.is_current_stream_capturing():
            return _new((need,), torch.uint8, dev), need
        key = (dev, _raw_stream(dev))
        mine = _kept.__dict__
        workspace = mine.pop(key, None)
        if workspace is None or workspace.numel() < need:
            workspace = _new((need,), torch.uint8, dev)
        mine[key] = workspace  # the latest one last
        if len(mine) > _KEPT_STREAMS:
            del mine[next(iter(mine))]
        return workspace, need
    _cuda(workspace, "workspace")
    if workspace.dtype != torch.uint8 or workspace.get_device() != dev:
        raise ValueError("workspace must be a uint8 tensor on cuda:%d" % dev)
    return workspace, workspace.numel()


def release_workspaces():
    """Gives back the workspaces that the binding keeps for the calling thread
    (up to 16 MB for each of the eight streams it used last; a thread's go with
    it when it ends)."""
    _kept.__dict__.clear()


def rms_norm_backward(dy, h, rstd, weight, dh=None, weight_grad=True, dx=None, dweight=None,
                      workspace=None):
    """fos_rms_norm_backward: (dx, dweight) from the gradient dy of the norm's
    output, the h and rstd the forward call returned, and optionally the
    gradient dh that reaches h from elsewhere.  dx is the gradient of x and of
    the residual, and may be passed as dy, h or dh; dweight is fp32 (None
    without weight_grad).  workspace: at least
    fos_rms_norm_backward_workspace_bytes of uint8; when None, one that the
    binding keeps for this thread and stream (up to 16 MB, else allocated; see
    release_workspaces)."""
    shape, dt, dev = _data(dy, "dy")
    R, C = shape
    _like(h, "h", shape, dy.dtype, dev)
    _like(rstd, "rstd", (R,), torch.float32, dev)
    wdt = _weight(weight, C, dy.dtype, dev)
    if dh is not None:
        _like(dh, "dh", shape, dy.dtype, dev)
    dx = torch.empty_like(dy) if dx is None else _like(dx, "dx", shape, dy.dtype, dev)
    nws = 0
    if weight_grad:
        if dweight is None:
            dweight = _new((C,), torch.float32, dev)
        else:
            _like(dweight, "dweight", (C,), torch.float32, dev)
        # fos_rms_norm_backward_workspace_bytes, without the call
        workspace, nws = _workspace(workspace, 0 if R <= 1 else min(R, 1024) * C * 4, dev)
    else:
        dweight = workspace = None
    _check(lib().fos_rms_norm_backward(dy.data_ptr(), h.data_ptr(), _a(dh), rstd.data_ptr(),
                                       weight.data_ptr(), dt, wdt, R, C, dx.data_ptr(),
                                       _a(dweight), _a(workspace), nws, _stream(dy)),
           "fos_rms_norm_backward")
    return dx, dweight


def quantize8(x, scale_tiled=True, rowwise=True, colwise=False, codes=None, scales=None,
              codes_t=None, scales_t=None):
    """fos_quantize8: x [rows, cols] in the 8-bit block format.  Returns
    (codes, scales, codes_t, scales_t); the first two are the rows of x (None
    without rowwise), the last two the rows of x.T padded with zeros to a
    multiple of 32 (None without colwise)."""
    (R, C), dt, dev = _data(x, "x")
    if rowwise:
        codes, scales = _pair8(R, C, scale_tiled, codes, scales, dev)
    else:
        codes = scales = None
    if colwise:
        codes_t, scales_t = _pair8(C, (R + 31) // 32 * 32, scale_tiled, codes_t, scales_t, dev,
                                   ("codes_t", "scales_t"))
    else:
        codes_t = scales_t = None
    _check(lib().fos_quantize8(x.data_ptr(), dt, R, C, 1 if scale_tiled else 0, _a(codes),
                               _a(scales), _a(codes_t), _a(scales_t), _stream(x)),
           "fos_quantize8")
    return codes, scales, codes_t, scales_t


def act_backward(dout, pre, act, scale_tiled=True, rowwise=True, colwise=True, value=False,
                 bias_grad=True, codes=None, scales=None, codes_t=None, scales_t=None, d=None,
                 dbias=None, workspace=None):
    """fos_act_backward: d = dout * act'(pre), as (codes, scales, codes_t,
    scales_t, d, dbias): its 8-bit rows (rowwise), its 8-bit columns
    (colwise), d itself (value) and the fp32 sum of its columns (bias_grad);
    what is not asked for is None.  act: "none", "relu", "gelu", "gelu_tanh",
    "silu"; pre may be None with "none".  d may be passed as dout or as pre.
    workspace: as in rms_norm_backward (fos_act_backward_workspace_bytes)."""
    shape, dt, dev = _data(dout, "dout")
    R, C = shape
    a = _act(act)
    if pre is not None:
        _like(pre, "pre", shape, dout.dtype, dev)
    if rowwise:
        codes, scales = _pair8(R, C, scale_tiled, codes, scales, dev)
    else:
        codes = scales = None
    if colwise:
        codes_t, scales_t = _pair8(C, (R + 31) // 32 * 32, scale_tiled, codes_t, scales_t, dev,
                                   ("codes_t", "scales_t"))
    else:
        codes_t = scales_t = None
    if value:
        d = torch.empty_like(dout) if d is None else _like(d, "d", shape, dout.dtype, dev)
    else:
        d = None
    nws = 0
    if bias_grad:
        if dbias is None:
            dbias = _new((C,), torch.float32, dev)
        else:
            _like(dbias, "dbias", (C,), torch.float32, dev)
        # fos_act_backward_workspace_bytes, without the call
        workspace, nws = _workspace(workspace, 0 if R <= 128 else (R + 127) // 128 * C * 4, dev)
    else:
        dbias = workspace = None
    _check(lib().fos_act_backward(dout.data_ptr(), _a(pre), dt, R, C, a, 1 if scale_tiled else 0,
                                  _a(d), _a(codes), _a(scales), _a(codes_t), _a(scales_t),
                                  _a(dbias), _a(workspace), nws, _stream(dout)),
           "fos_act_backward")
    return codes, scales, codes_t, scales_t, d, dbias


def _operand(codes, scales, name, blk, dev=None):
    """Checks a product operand's codes [rows, bytes] and flat tiled scales
    (blk elements per scale, 32 / blk elements per byte)."""
    if not isinstance(codes, torch.Tensor) or not codes.is_cuda or not codes.is_contiguous():
        _cuda(codes, name + "_codes")
    on = codes.get_device()
    shape = codes.shape
    if len(shape) != 2 or codes.dtype is not torch.uint8 or (dev is not None and on != dev):
        raise ValueError("%s_codes must be a rank-2 uint8 tensor on the product's device" % name)
    R, K = shape[0], shape[1] * (32 // blk)
    if scales.dtype is not torch.uint8 or scales.get_device() != on or \
            not scales.is_contiguous() or \
            scales.numel() != (R + 127) // 128 * ((K + 4 * blk - 1) // (4 * blk)) * 512:
        raise ValueError("%s_scales must be the tiled uint8 scales of %s_codes" % (name, name))
    return R, K, on


def _epilogue(M, N, act, bias, residual, out_dtype, save_pre, out, pre, dev):
    if out_dtype not in _DT:
        raise ValueError("out_dtype must be bf16, fp16 or fp32")
    if bias is not None:
        if bias.dtype not in (torch.float32, out_dtype):
            raise ValueError("bias must be float32 or of the output's type")
        _like(bias, "bias", (N,), bias.dtype, dev)
    if residual is not None:
        _like(residual, "residual", (M, N), out_dtype, dev)
    if out is None:
        out = _new((M, N), out_dtype, dev)
    else:
        _like(out, "out", (M, N), out_dtype, dev)
    if not save_pre:
        pre = None
    elif pre is None:
        pre = _new((M, N), out_dtype, dev)
    else:
        _like(pre, "pre", (M, N), out_dtype, dev)
    return FosEpilogue(_act(act), _DT[out_dtype], _DT[bias.dtype] if bias is not None else FOS_FP32,
                       _a(bias), _a(residual), _a(pre)), out, pre


def linear8(a_codes, a_scales, b_codes, b_scales, act="none", bias=None, residual=None,
            out_dtype=torch.bfloat16, save_pre=False, out=None, pre=None):
    """fos_linear8: act(a . b^T + bias) + residual from 8-bit block operands a
    [M, K] and b [N, K] (codes, tiled scales).  bias [N] is fp32 or of the
    output's type, residual [M, N] of the output's type; out may be the residual
    itself.  Returns out, or (out, pre) with save_pre: pre is the value before
    the activation, which act_backward reads."""
    M, K, dev = _operand(a_codes, a_scales, "a", 32)
    N, Kb, _ = _operand(b_codes, b_scales, "b", 32, dev)
    if K != Kb:
        raise ValueError("a and b must have the same K")
    ep, out, pre = _epilogue(M, N, act, bias, residual, out_dtype, save_pre, out, pre, dev)
    _check(lib().fos_linear8(a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(),
                             b_scales.data_ptr(), M, N, K, ctypes.byref(ep), out.data_ptr(),
                             _stream(a_codes)), "fos_linear8")
    return (out, pre) if save_pre else out


def linear4(a_codes, a_scales, a_amax, b_codes, b_scales, b_amax, act="none", bias=None,
            residual=None, out_dtype=torch.bfloat16, save_pre=False, cfg=Config(), out=None,
            pre=None):
    """fos_linear4: linear8 for NVFP4 operands (1x16 codes, tiled scales, and
    the amaxes they were quantized with; cfg.row_scaled when a has one per row)."""
    M, K, dev = _operand(a_codes, a_scales, "a", 16)
    N, Kb, _ = _operand(b_codes, b_scales, "b", 16, dev)
    if K != Kb:
        raise ValueError("a and b must have the same K")
    _like(a_amax, "a_amax", (M if cfg.row_scaled else 1,), torch.float32, dev)
    _like(b_amax, "b_amax", (1,), torch.float32, dev)
    ep, out, pre = _epilogue(M, N, act, bias, residual, out_dtype, save_pre, out, pre, dev)
    cc = cfg.c(True)
    _check(lib().fos_linear4(a_codes.data_ptr(), a_scales.data_ptr(), a_amax.data_ptr(),
                             b_codes.data_ptr(), b_scales.data_ptr(), b_amax.data_ptr(), M, N, K,
                             ctypes.byref(cc), ctypes.byref(ep), out.data_ptr(),
                             _stream(a_codes)), "fos_linear4")
    return (out, pre) if save_pre else out


# ------------------------------------------------------------------ by expert
def _ends(offs, dev, name="offs"):
    """Checks the experts' cumulative ends (or the rows' experts); returns their number."""
    if not isinstance(offs, torch.Tensor) or offs.dtype is not torch.int32 or offs.dim() != 1 or \
            offs.get_device() != dev or not offs.is_contiguous():
        raise ValueError("%s must be a contiguous int32 vector on cuda:%d" % (name, dev))
    return offs.shape[0]


def _experts(codes, scales, name, G, blk, dev):
    """Checks the experts' weights: codes [G, N, bytes] and each one's flat tiled
    scales one after the other; returns (N, K)."""
    if not isinstance(codes, torch.Tensor) or codes.dtype is not torch.uint8 or codes.dim() != 3 or \
            codes.shape[0] != G or codes.get_device() != dev or not codes.is_contiguous():
        raise ValueError("%s_codes must be a contiguous uint8 tensor [%d, N, bytes] on cuda:%d"
                         % (name, G, dev))
    N, K = codes.shape[1], codes.shape[2] * (32 // blk)
    if scales.dtype is not torch.uint8 or scales.get_device() != dev or not scales.is_contiguous() or \
            scales.numel() != G * ((N + 127) // 128) * ((K + 4 * blk - 1) // (4 * blk)) * 512:
        raise ValueError("%s_scales must be the tiled uint8 scales of every expert's %s_codes"
                         % (name, name))
    return N, K


def _packed(codes, scales, blk):
    """Checks packed rows' codes [rows, bytes] and plain scales; returns (rows, K, device)."""
    if not isinstance(codes, torch.Tensor) or not codes.is_cuda or not codes.is_contiguous():
        _cuda(codes, "a_codes")
    dev = codes.get_device()
    if codes.dim() != 2 or codes.dtype is not torch.uint8:
        raise ValueError("a_codes must be a rank-2 uint8 tensor")
    R, K = codes.shape[0], codes.shape[1] * (32 // blk)
    _like(scales, "a_scales", (R, K // blk), torch.uint8, dev)
    return R, K, dev


def _grouped_epilogue(G, M, N, act, bias, residual, out_dtype, save_pre, out, pre, dev):
    """_epilogue() with a bias row an expert."""
    if bias is not None:
        if bias.dtype not in (torch.float32, out_dtype):
            raise ValueError("bias must be float32 or of the output's type")
        _like(bias, "bias", (G, N), bias.dtype, dev)
    ep, out, pre = _epilogue(M, N, act, None, residual, out_dtype, save_pre, out, pre, dev)
    if bias is not None:
        ep.bias_dt, ep.bias = _DT[bias.dtype], bias.data_ptr()
    return ep, out, pre


def linear8_grouped(a_codes, a_scales, b_codes, b_scales, offs, act="none", bias=None, residual=None,
                    out_dtype=torch.bfloat16, save_pre=False, out=None, pre=None):
    """fos_linear8_grouped: act(a . b[e]^T + bias[e]) + residual, e the expert of
    each row of a.  a: packed rows' codes [M, K] and plain scales [M, K/32];
    b: the experts' codes [G, N, K] and their tiled scales; offs: int32 [G],
    cumulative ends.  bias [G, N], residual [M, N]; out may be the residual itself.
    Rows past the last end keep what out (and pre) hold.  Returns out, or (out,
    pre) with save_pre."""
    M, K, dev = _packed(a_codes, a_scales, 32)
    G = _ends(offs, dev)
    N, Kb = _experts(b_codes, b_scales, "b", G, 32, dev)
    if K != Kb:
        raise ValueError("a and b must have the same K")
    ep, out, pre = _grouped_epilogue(G, M, N, act, bias, residual, out_dtype, save_pre, out, pre, dev)
    _check(lib().fos_linear8_grouped(a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(),
                                     b_scales.data_ptr(), offs.data_ptr(), G, M, N, K,
                                     ctypes.byref(ep), out.data_ptr(), _stream(a_codes)),
           "fos_linear8_grouped")
    return (out, pre) if save_pre else out


def linear4_grouped(a_codes, a_scales, a_amax, b_codes, b_scales, b_amax, offs, act="none", bias=None,
                    residual=None, out_dtype=torch.bfloat16, save_pre=False, cfg=Config(), out=None,
                    pre=None):
    """fos_linear4_grouped: linear8_grouped for NVFP4 operands: what
    quantize_grouped returns for the packed rows (a_amax [G]; [M] with
    cfg.row_scaled), the experts' codes [G, N, K/2], their tiled scales and
    b_amax [G]."""
    M, K, dev = _packed(a_codes, a_scales, 16)
    G = _ends(offs, dev)
    N, Kb = _experts(b_codes, b_scales, "b", G, 16, dev)
    if K != Kb:
        raise ValueError("a and b must have the same K")
    _like(a_amax, "a_amax", (M if cfg.row_scaled else G,), torch.float32, dev)
    _like(b_amax, "b_amax", (G,), torch.float32, dev)
    ep, out, pre = _grouped_epilogue(G, M, N, act, bias, residual, out_dtype, save_pre, out, pre, dev)
    cc = cfg.c(True)
    _check(lib().fos_linear4_grouped(a_codes.data_ptr(), a_scales.data_ptr(), a_amax.data_ptr(),
                                     b_codes.data_ptr(), b_scales.data_ptr(), b_amax.data_ptr(),
                                     offs.data_ptr(), G, M, N, K, ctypes.byref(cc),
                                     ctypes.byref(ep), out.data_ptr(), _stream(a_codes)),
           "fos_linear4_grouped")
    return (out, pre) if save_pre else out


def grouped_cols(rows, groups):
    """Columns of the column-wise form of `rows` packed rows: every expert's part
    padded to a multiple of 128, for any routing."""
    n = lib().fos_grouped_cols(int(rows), int(groups))
    if n < 0:
        raise ValueError("bad number of rows or experts")
    return n


def quantize8_grouped(x, offs, rowwise=True, colwise=True, codes=None, scales=None, codes_t=None,
                      scales_t=None):
    """fos_quantize8_grouped: packed rows x [rows, cols] in the 8-bit block format.
    Returns (codes, scales, codes_t, scales_t): the rows with plain scales [rows,
    cols/32] (None without rowwise) and, with grouped_cols(rows, G) columns, the
    rows of x.T, each expert's part padded with zeros to a multiple of 128, with
    tiled scales (None without colwise)."""
    (R, C), dt, dev = _data(x, "x")
    G = _ends(offs, dev)
    codes, scales = _pair8(R, C, False, codes, scales, dev) if rowwise else (None, None)
    codes_t, scales_t = _pair8(C, grouped_cols(R, G), True, codes_t, scales_t, dev,
                               ("codes_t", "scales_t")) if colwise else (None, None)
    _check(lib().fos_quantize8_grouped(x.data_ptr(), dt, R, C, offs.data_ptr(), G, _a(codes),
                                       _a(scales), _a(codes_t), _a(scales_t), _stream(x)),
           "fos_quantize8_grouped")
    return codes, scales, codes_t, scales_t


def act_backward_grouped(dout, pre, act, offs, rowwise=True, colwise=True, value=False,
                         bias_grad=True, codes=None, scales=None, codes_t=None, scales_t=None,
                         d=None, dbias=None, workspace=None):
    """fos_act_backward_grouped: act_backward of packed rows, as (codes, scales,
    codes_t, scales_t, d, dbias): the 8-bit forms as in quantize8_grouped, d with
    value, and dbias [G, cols], the sum of each expert's rows.  d may be passed as
    dout or as pre.  workspace: as in rms_norm_backward
    (fos_act_backward_grouped_workspace_bytes)."""
    shape, dt, dev = _data(dout, "dout")
    R, C = shape
    a = _act(act)
    G = _ends(offs, dev)
    if pre is not None:
        _like(pre, "pre", shape, dout.dtype, dev)
    P = grouped_cols(R, G)
    codes, scales = _pair8(R, C, False, codes, scales, dev) if rowwise else (None, None)
    codes_t, scales_t = _pair8(C, P, True, codes_t, scales_t, dev,
                               ("codes_t", "scales_t")) if colwise else (None, None)
    if value:
        d = torch.empty_like(dout) if d is None else _like(d, "d", shape, dout.dtype, dev)
    else:
        d = None
    nws = 0
    if bias_grad:
        if dbias is None:
            dbias = _new((G, C), torch.float32, dev)
        else:
            _like(dbias, "dbias", (G, C), torch.float32, dev)
        # fos_act_backward_grouped_workspace_bytes, without the call
        workspace, nws = _workspace(workspace, 0 if R == 0 else 4 * (P // 128 * C + G + 1), dev)
    else:
        dbias = workspace = None
    _check(lib().fos_act_backward_grouped(dout.data_ptr(), _a(pre), dt, R, C, offs.data_ptr(), G, a,
                                          _a(d), _a(codes), _a(scales), _a(codes_t), _a(scales_t),
                                          _a(dbias), _a(workspace), nws, _stream(dout)),
           "fos_act_backward_grouped")
    return codes, scales, codes_t, scales_t, d, dbias


def linear8_grouped_wgrad(d_codes_t, d_scales_t, z_codes_t, z_scales_t, offs, rows, residual=None,
                          out_dtype=torch.float32, out=None):
    """fos_linear8_grouped_wgrad: the experts' weight gradients [G, N, K], d^T . z
    over each expert's rows (+ residual), from the column-wise forms of d [rows, N]
    and z [rows, K] that quantize8_grouped and act_backward_grouped return for the
    same offs.  An expert without rows gets its residual, or zeros.  out may be the
    residual itself."""
    N, P, dev = _operand(d_codes_t, d_scales_t, "d", 32)
    K, Pz, _ = _operand(z_codes_t, z_scales_t, "z", 32, dev)
    G = _ends(offs, dev)
    if P != Pz or P != grouped_cols(rows, G):
        raise ValueError("d and z must have grouped_cols(rows, %d) columns" % G)
    if out_dtype not in _DT:
        raise ValueError("out_dtype must be bf16, fp16 or fp32")
    if residual is not None:
        _like(residual, "residual", (G, N, K), out_dtype, dev)
    out = _new((G, N, K), out_dtype, dev) if out is None else _like(out, "out", (G, N, K), out_dtype, dev)
    _check(lib().fos_linear8_grouped_wgrad(d_codes_t.data_ptr(), d_scales_t.data_ptr(),
                                           z_codes_t.data_ptr(), z_scales_t.data_ptr(),
                                           offs.data_ptr(), G, rows, N, K, _a(residual),
                                           _DT[out_dtype], out.data_ptr(), _stream(d_codes_t)),
           "fos_linear8_grouped_wgrad")
    return out


def matvec4(x, b_codes, b_scales, b_amax, ids=None, act="none", bias=None, residual=None,
            out_dtype=None, cfg=Config(), out=None):
    """fos_matvec4: act(x . b[e]^T + bias[e]) + residual for few rows x [X, K] that
    stay in bf16, fp16 or fp32 (no element is rounded), with NVFP4 weights; for 16
    rows and more (4 of fp32) linear4 of quantized rows takes less.  Without ids b is one matrix
    (codes [N, K/2], tiled scales, amax [1], bias [N]); with ids (int32 [M], M a
    multiple of X) row p takes x[p // (M / X)] and expert ids[p] of codes [G, N,
    K/2], their tiled scales, amax [G], bias [G, N]; a row with an id outside 0 ..
    G - 1 keeps what out holds.  out and residual [M, N] are of out_dtype (x's own
    by default); out may be the residual itself."""
    (X, K), dt, dev = _data(x, "x")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    if ids is None:
        M, G = X, 1
        N, Kb, _ = _operand(b_codes, b_scales, "b", 16, dev)
        ep, out, _ = _epilogue(M, N, act, bias, residual, out_dtype, False, out, None, dev)
    else:
        M, G = _ends(ids, dev, "ids"), b_codes.shape[0]
        N, Kb = _experts(b_codes, b_scales, "b", G, 16, dev)
        ep, out, _ = _grouped_epilogue(G, M, N, act, bias, residual, out_dtype, False, out, None, dev)
    if K != Kb:
        raise ValueError("x and b must have the same K")
    _like(b_amax, "b_amax", (G,), torch.float32, dev)
    cc = cfg.c(True)
    _check(lib().fos_matvec4(x.data_ptr(), dt, X, _a(ids), b_codes.data_ptr(), b_scales.data_ptr(),
                             b_amax.data_ptr(), M, N, K, G, ctypes.byref(cc), ctypes.byref(ep),
                             out.data_ptr(), _stream(x)), "fos_matvec4")
    return out


DIAG_E2M1_ENCODE, DIAG_E2M1_DECODE, DIAG_E4M3_ENCODE, DIAG_E4M3_DECODE = 0, 1, 2, 3
DIAG_F16_ROUND, DIAG_BF16_BITS, DIAG_F16_BITS, DIAG_DIV6 = 4, 5, 6, 7
DIAG_SCALE_CODES = 8


def diag_convert(op, inp, out):
    """Element-wise access to one device conversion primitive (fos_diag.h)."""
    _cuda(inp, "inp")
    _cuda(out, "out")
    _check(lib().fos_diag_convert(int(op), _p(inp), _p(out), inp.numel(), _stream(inp)),
           "fos_diag_convert")
    return out
