"""The feed-forward operators without a GPU: sizes of their buffers, argument
checks of the C entry points (every call below stops on the host), and the
binding's refusal of tensors that are not on a CUDA device."""
import ctypes
import random

import pytest
import torch

import ffn_reference as ref
import nvfp4_quantization_precision_gb300 as fos
from nvfp4_quantization_precision_gb300 import build as fos_build

I64 = ctypes.c_int64
FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced
ODD = ctypes.c_void_p(0x10010)   # 16-byte, not 32-byte aligned
INV, UNS, MIS = fos.FOS_ERR_INVALID_ARG, fos.FOS_ERR_UNSUPPORTED, fos.FOS_ERR_MISALIGNED


@pytest.fixture(scope="module")
def L():
    fos_build.build()
    return fos.lib()


def test_scales8_bytes(L):
    for rows, cols in [(1, 32), (128, 128), (129, 160), (300, 4096)]:
        assert L.fos_scales8_bytes(rows, cols, 0) == rows * cols // 32
        n = L.fos_scales8_bytes(rows, cols, 1)
        assert n == -(-rows // 128) * -(-cols // 128) * 512
        assert int(ref.tile_index(rows, cols // 32).max()) < n
        assert fos.scales8_shape(rows, cols) == (n,)
        assert fos.scales8_shape(rows, cols, False) == (rows, cols // 32)
    for rows, cols, layout in [(-1, 32, 0), (1, 16, 0), (1, -32, 1), (1, 32, 2)]:
        assert L.fos_scales8_bytes(rows, cols, layout) == -1
    with pytest.raises(ValueError):
        fos.scales8_shape(4, 48)


def test_workspace_bytes(L):
    f, g = L.fos_rms_norm_backward_workspace_bytes, L.fos_act_backward_workspace_bytes
    assert f(0, 64) == f(1, 64) == 0 and f(2, 64) == 512 and f(10 ** 6, 64) == 1024 * 256
    assert g(128, 64) == 0 and g(129, 64) == 512 and g(1000, 64) == 8 * 256


def _norm(L, x=FAKE, res=None, w=FAKE, dt=0, wdt=2, rows=4, cols=64, eps=1e-6, layout=1, h=None,
          y=None, codes=FAKE, scales=FAKE, rstd=FAKE):
    return L.fos_rms_norm(x, res, w, dt, wdt, rows, cols, eps, layout, h, y, codes, scales, rstd, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(dt=5), INV), (dict(dt=0, wdt=1), INV), (dict(rows=-1), INV), (dict(cols=48), UNS),
    (dict(cols=0), UNS), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(layout=2), INV), (dict(x=None), INV), (dict(w=None), INV),
    (dict(codes=None), INV), (dict(scales=None), INV), (dict(x=ODD), MIS), (dict(res=ODD), MIS),
    (dict(h=ODD), MIS), (dict(y=ODD), MIS), (dict(codes=ctypes.c_void_p(0x10008)), MIS),
    (dict(scales=ctypes.c_void_p(0x10002)), MIS), (dict(rstd=ctypes.c_void_p(0x10002)), MIS),
    (dict(rows=1 << 31), UNS), (dict(rows=1 << 29, cols=1 << 20), UNS), (dict(rows=0), fos.FOS_OK),
    (dict(codes=None, scales=None, rstd=None), INV)])
def test_rms_norm_checks(L, kw, rc):
    assert _norm(L, **kw) == rc


def _back(L, dy=FAKE, h=FAKE, dh=None, rstd=FAKE, w=FAKE, dt=0, wdt=2, rows=4, cols=64, dx=FAKE,
          dw=FAKE, ws=FAKE, n=1 << 20):
    return L.fos_rms_norm_backward(dy, h, dh, rstd, w, dt, wdt, rows, cols, dx, dw, ws, n, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(dy=None), INV), (dict(dx=None), INV), (dict(rstd=None), INV), (dict(ws=None), INV),
    (dict(n=16), INV), (dict(ws=ODD), MIS), (dict(dy=ODD), MIS), (dict(dw=ODD), MIS),
    (dict(cols=40), UNS), (dict(wdt=1), INV), (dict(cols=0), UNS),
    (dict(rows=0, dw=None), fos.FOS_OK)])
def test_rms_norm_backward_checks(L, kw, rc):
    assert _back(L, **kw) == rc


def _quant(L, x=FAKE, dt=0, rows=4, cols=64, layout=1, c=FAKE, s=FAKE, ct=None, st=None):
    return L.fos_quantize8(x, dt, rows, cols, layout, c, s, ct, st, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(dt=3), INV), (dict(cols=16), UNS), (dict(rows=-4), INV), (dict(layout=7), INV),
    (dict(x=None), INV), (dict(c=None), INV), (dict(c=None, s=None), INV), (dict(ct=FAKE), INV),
    (dict(ct=ODD, st=FAKE), MIS), (dict(x=ODD), MIS), (dict(rows=0), fos.FOS_OK),
    (dict(cols=0), fos.FOS_OK)])
def test_quantize8_checks(L, kw, rc):
    assert _quant(L, **kw) == rc


def test_act_backward_checks(L):
    def call(dout=FAKE, pre=FAKE, act=4, rows=200, dbias=None, ws=None, n=0, d=FAKE):
        return L.fos_act_backward(dout, pre, 0, rows, 64, act, 1, d, None, None, None, None, dbias,
                                  ws, n, None)
    assert call(act=5) == INV and call(act=-1) == INV and call(pre=None) == INV
    assert call(dbias=FAKE) == INV and call(dbias=FAKE, ws=FAKE, n=100) == INV
    assert call(dbias=FAKE, ws=ODD, n=1 << 20) == MIS and call(d=ODD) == MIS
    assert call(d=None) == INV


def _ep(act=0, out_dt=0, bias_dt=2, bias=None, residual=None, pre=None):
    return fos.FosEpilogue(act, out_dt, bias_dt, bias, residual, pre)


@pytest.mark.parametrize("kw,rc", [
    (dict(M=-1), INV), (dict(N=24), UNS), (dict(K=48), UNS), (dict(K=0), UNS), (dict(a=None), INV),
    (dict(out=None), INV), (dict(a=ctypes.c_void_p(0x10008)), MIS),
    (dict(out=ctypes.c_void_p(0x10008)), MIS), (dict(ep=_ep(act=9)), INV),
    (dict(ep=_ep(out_dt=3)), INV), (dict(ep=_ep(bias_dt=1, bias=0x10000)), INV),
    (dict(ep=_ep(bias=0x10004)), MIS), (dict(ep=_ep(residual=0x10008)), MIS), (dict(ep=None), INV),
    (dict(M=0), fos.FOS_OK), (dict(N=0), fos.FOS_OK), (dict(M=1 << 30), UNS),
    (dict(M=1 << 25, K=1 << 20), UNS)])
def test_linear_checks(L, kw, rc):
    p = dict(a=FAKE, M=4, N=64, K=128, ep=_ep(), out=FAKE)
    p.update(kw)
    ep = ctypes.byref(p["ep"]) if p["ep"] is not None else None
    assert L.fos_linear8(p["a"], FAKE, FAKE, FAKE, p["M"], p["N"], p["K"], ep, p["out"], None) == rc
    cfg = fos.Config().c(True)
    assert L.fos_linear4(p["a"], FAKE, FAKE, FAKE, FAKE, FAKE, p["M"], p["N"], p["K"],
                         ctypes.byref(cfg), ep, p["out"], None) == rc


def test_linear4_checks_its_config(L):
    ep = _ep()
    for cfg, rc in ((fos.Config(block16x16=True).c(True), UNS), (fos.Config(bound=300).c(True), UNS)):
        assert L.fos_linear4(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 128, ctypes.byref(cfg),
                             ctypes.byref(ep), FAKE, None) == rc
    assert L.fos_linear4(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 128, None, ctypes.byref(ep),
                         FAKE, None) == INV
    cfg = fos.Config().c(True)
    assert L.fos_linear4(FAKE, FAKE, None, FAKE, FAKE, FAKE, 4, 64, 128, ctypes.byref(cfg),
                         ctypes.byref(ep), FAKE, None) == INV


def test_random_arguments_never_crash(L):
    """Seeded random sizes, enums and pointers: each call returns a status; with
    no GPU, what passes the checks stops at the pointer check."""
    rng = random.Random(77)
    sizes = [-32, -1, 0, 1, 31, 32, 64, 100, 4096, 1 << 29, 1 << 31, 1 << 40, 1 << 62]
    ptrs = [None, FAKE, ODD, ctypes.c_void_p(0x10001)]
    for _ in range(600):
        p = [rng.choice(ptrs) for _ in range(9)]
        R, C, K = (I64(rng.choice(sizes)) for _ in range(3))
        dt, e = rng.choice([0, 1, 2, 7]), rng.choice([0, 1, 2, 4, 9])
        ep = _ep(e, dt, rng.choice([0, 2, 5]), rng.choice([None, 0x10000, 0x10004]))
        cfg = fos.Config(row_scaled=rng.random() < 0.5).c(True)
        n = rng.choice([0, 512, 1 << 30])
        rcs = [
            L.fos_rms_norm(p[0], p[1], p[2], dt, 2, R, C, 1e-6, rng.choice([0, 1, 2]), p[3], p[4], p[5],
                           p[6], p[7], None),
            L.fos_rms_norm_backward(p[0], p[1], p[2], p[3], p[4], dt, 2, R, C, p[5], p[6], p[7], n, None),
            L.fos_quantize8(p[0], dt, R, C, 1, p[1], p[2], p[3], p[4], None),
            L.fos_act_backward(p[0], p[1], dt, R, C, e, 0, p[2], p[3], p[4], p[5], p[6], p[7], p[8], n,
                               None),
            L.fos_linear8(p[0], p[1], p[2], p[3], R, C, K, ctypes.byref(ep), p[4], None),
            L.fos_linear4(p[0], p[1], p[2], p[3], p[4], p[5], R, C, K, ctypes.byref(cfg),
                          ctypes.byref(ep), p[6], None)]
        assert all(rc in range(6) for rc in rcs), rcs


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(4, 64), torch.ones(64)
    u8 = torch.zeros(4, 64, dtype=torch.uint8)
    for f in (lambda: fos.rms_norm(x, w), lambda: fos.quantize8(x),
              lambda: fos.rms_norm_backward(x, x, torch.ones(4), w),
              lambda: fos.act_backward(x, x, "gelu"), lambda: fos.linear8(u8, u8, u8, u8),
              lambda: fos.linear4(u8, u8, x, u8, u8, x)):
        with pytest.raises(ValueError):
            f()


def test_reference_forms_agree_with_each_other():
    """The 64-bit forms the GPU tests use: code and scale round trips, the tiled
    index as a bijection, derivatives against differences."""
    v = torch.randn(7, 96, dtype=torch.float64, generator=torch.Generator().manual_seed(1)) * 3
    q, s = ref.quantize8(v)
    back = ref.blocks(q) * ref.pow2(s - 127).unsqueeze(2)
    assert ((back - ref.blocks(v)).abs() <= ref.blocks(v).abs() / 16 + ref.pow2(s - 127).unsqueeze(2) * 2.0 ** -10).all()
    assert (ref.amax_of(v) <= 448 * ref.pow2(s - 127)).all()
    assert (ref.amax_of(v) > 448 * ref.pow2(s - 128)).all()
    idx = ref.tile_index(300, 9)
    assert idx.unique().numel() == idx.numel()
    p = torch.linspace(-5, 5, 501, dtype=torch.float64) + 1e-3
    for a in ("relu", "gelu", "gelu_tanh", "silu"):
        num = (ref.act(p + 1e-5, a) - ref.act(p - 1e-5, a)) / 2e-5
        assert (num - ref.act_slope(p, a)).abs().max() < 1e-8
