"""The operators on rows packed by expert without a GPU: sizes of their buffers,
argument checks of the C entry points (every call below stops on the host), the
binding's refusal of tensors that are not on a CUDA device, and rules of their
kernels read from the source."""
import ctypes
import os
import random
import re

import pytest
import torch

import expert_reference as ex
import nvfp4_quantization_precision_gb300 as fos
from nvfp4_quantization_precision_gb300 import build as fos_build

FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced
ODD = ctypes.c_void_p(0x10008)
INV, UNS, MIS, OK = fos.FOS_ERR_INVALID_ARG, fos.FOS_ERR_UNSUPPORTED, fos.FOS_ERR_MISALIGNED, fos.FOS_OK


@pytest.fixture(scope="module")
def L():
    fos_build.build()
    return fos.lib()


def test_grouped_cols(L):
    """Room for every routing: no split of the rows needs more, some split needs all."""
    r = random.Random(1)
    for _ in range(300):
        rows, G = r.randrange(0, 2000), r.randrange(1, 40)
        P = L.fos_grouped_cols(rows, G)
        assert P == ex.columns(rows, G)
        offs = sorted(r.randrange(0, rows + 1) for _ in range(G))
        assert ex.spans(offs, rows)[-1][4] <= P
    # one row each but the last: the most
    for rows, G in ((7, 20), (300, 3), (129, 2), (128, 1)):
        n = min(G, rows)
        offs = list(range(1, n)) + [rows] * (G - n + 1)
        assert ex.spans(offs, rows)[-1][4] in (L.fos_grouped_cols(rows, G), L.fos_grouped_cols(rows, G) - 128)
    for rows, G in ((-1, 4), (4, 0), (4, -1), (4, 1025), (1 << 62, 4)):
        assert L.fos_grouped_cols(rows, G) == -1
        with pytest.raises(ValueError):
            fos.grouped_cols(rows, min(G, 2000)) if rows < 1 << 62 else fos.grouped_cols(rows, G)


def test_workspace_bytes(L):
    f = L.fos_act_backward_grouped_workspace_bytes
    assert f(0, 64, 4) == f(10, 0, 4) == f(10, 48, 4) == f(10, 64, 0) == f(10, 64, 1025) == 0
    assert f(300, 64, 3) == (ex.columns(300, 3) // 128 * 64 + 4) * 4
    for rows, cols in ((1 << 62, 32), (32, 1 << 62), (1 << 40, 1 << 40)):
        assert f(rows, cols, 8) == 0


def _ep(act=0, out_dt=0, bias_dt=2, bias=None, residual=None, pre=None):
    return fos.FosEpilogue(act, out_dt, bias_dt, bias, residual, pre)


@pytest.mark.parametrize("kw,rc", [
    (dict(rows=-1), INV), (dict(N=-16), INV), (dict(N=24), UNS), (dict(K=96), UNS), (dict(K=0), UNS),
    (dict(G=0), INV), (dict(G=-3), INV), (dict(G=1025), UNS), (dict(a=None), INV), (dict(s=None), INV),
    (dict(offs=None), INV), (dict(out=None), INV), (dict(a=ODD), MIS), (dict(s=ODD), MIS),
    (dict(offs=ctypes.c_void_p(0x10002)), MIS), (dict(out=ODD), MIS), (dict(ep=None), INV),
    (dict(ep=_ep(act=9)), INV), (dict(ep=_ep(out_dt=3)), INV), (dict(ep=_ep(bias_dt=1, bias=0x10000)), INV),
    (dict(ep=_ep(bias=0x10004)), MIS), (dict(ep=_ep(residual=0x10008)), MIS), (dict(rows=0), OK), (dict(N=0), OK),
    (dict(rows=1 << 30), UNS), (dict(rows=1 << 25, K=1 << 20), UNS), (dict(G=1024, N=1 << 21), UNS),
    (dict(G=1000, N=1 << 16, K=1 << 16), UNS)])
def test_grouped_products(L, kw, rc):
    p = dict(a=FAKE, s=FAKE, offs=FAKE, G=4, rows=9, N=64, K=128, ep=_ep(), out=FAKE)
    p.update(kw)
    ep = ctypes.byref(p["ep"]) if p["ep"] is not None else None
    size = (p["offs"], p["G"], p["rows"], p["N"], p["K"])
    assert L.fos_linear8_grouped(p["a"], p["s"], FAKE, FAKE, *size, ep, p["out"], None) == rc
    cfg = fos.Config().c(True)
    if kw.get("K") != 96:  # 96 = 64 + 32
        assert L.fos_linear4_grouped(p["a"], p["s"], FAKE, FAKE, FAKE, FAKE, *size, ctypes.byref(cfg), ep,
                                     p["out"], None) == rc


def test_grouped_nvfp4_configurations(L):
    def call(cfg, am=FAKE, bm=FAKE, K=64):
        ep = _ep()
        return L.fos_linear4_grouped(FAKE, FAKE, am, FAKE, FAKE, bm, FAKE, 2, 4, 64, K,
                                     ctypes.byref(cfg) if cfg else None, ctypes.byref(ep), FAKE, None)
    assert call(None) == INV
    assert call(fos.Config(block16x16=True).c(True)) == UNS
    assert call(fos.Config(bound=100).c(True)) == UNS
    bad = fos.Config().c(True)
    bad.granularity = 5
    assert call(bad) == INV
    assert call(fos.Config().c(True), am=None) == INV and call(fos.Config().c(True), bm=None) == INV
    assert call(fos.Config().c(True), K=32) == UNS


@pytest.mark.parametrize("kw,rc", [
    (dict(dt=3), INV), (dict(rows=-1), INV), (dict(cols=48), UNS), (dict(G=0), INV), (dict(G=1025), UNS),
    (dict(x=None), INV), (dict(offs=None), INV), (dict(c=None), INV), (dict(ct=None), INV),
    (dict(c=None, s=None, ct=None, st=None), INV), (dict(x=ctypes.c_void_p(0x10010)), MIS),
    (dict(ct=ctypes.c_void_p(0x10010)), MIS), (dict(c=ODD), MIS), (dict(st=ctypes.c_void_p(0x10002)), MIS),
    (dict(rows=0), OK), (dict(cols=0), OK), (dict(rows=(1 << 30) - 1, G=1024), UNS),
    (dict(rows=1 << 29, cols=1 << 20), UNS)])
def test_quantize8_grouped(L, kw, rc):
    p = dict(x=FAKE, dt=0, rows=9, cols=64, offs=FAKE, G=2, c=FAKE, s=FAKE, ct=FAKE, st=FAKE)
    p.update(kw)
    assert L.fos_quantize8_grouped(*[p[k] for k in ("x", "dt", "rows", "cols", "offs", "G", "c", "s", "ct", "st")],
                                   None) == rc


def test_act_backward_grouped(L):
    def call(pre=FAKE, act=4, rows=200, db=None, ws=None, n=0, d=FAKE, dout=FAKE):
        return L.fos_act_backward_grouped(dout, pre, 0, rows, 64, FAKE, 3, act, d, None, None, None, None, db, ws,
                                          n, None)
    assert call(act=5) == INV and call(pre=None) == INV and call(d=None) == INV and call(dout=None) == INV
    assert call(db=FAKE) == INV and call(db=FAKE, ws=FAKE, n=100) == INV
    assert call(db=FAKE, ws=ctypes.c_void_p(0x10010), n=1 << 20) == MIS
    assert call(rows=0) == OK


@pytest.mark.parametrize("kw,rc", [
    (dict(rows=-1), INV), (dict(N=24), UNS), (dict(K=40), UNS), (dict(K=0), UNS), (dict(G=0), INV),
    (dict(G=1025), UNS), (dict(dt=7), INV), (dict(d=None), INV), (dict(offs=None), INV), (dict(out=None), INV),
    (dict(d=ODD), MIS), (dict(out=ODD), MIS), (dict(res=ODD), MIS), (dict(N=0), OK), (dict(rows=1 << 30), UNS),
    (dict(G=1024, N=1 << 21), UNS), (dict(N=1 << 20, K=1 << 20, G=2), UNS)])
def test_wgrad(L, kw, rc):
    p = dict(d=FAKE, offs=FAKE, G=3, rows=50, N=64, K=32, res=None, dt=2, out=FAKE)
    p.update(kw)
    assert L.fos_linear8_grouped_wgrad(p["d"], FAKE, FAKE, FAKE, p["offs"], p["G"], p["rows"], p["N"], p["K"],
                                       p["res"], p["dt"], p["out"], None) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(dt=3), INV), (dict(M=-1), INV), (dict(N=24), UNS), (dict(K=48), UNS), (dict(K=0), UNS),
    (dict(M=1025), UNS), (dict(G=0), INV), (dict(G=2, ids=None), INV), (dict(G=1025), UNS), (dict(X=0), INV),
    (dict(X=3), INV), (dict(x=None), INV), (dict(out=None), INV), (dict(x=ODD), MIS), (dict(out=ODD), MIS),
    (dict(ids=ctypes.c_void_p(0x10002)), MIS), (dict(ep=_ep(pre=0x10000)), UNS), (dict(ep=None), INV),
    (dict(ep=_ep(act=-1)), INV), (dict(ep=_ep(bias=0x10004)), MIS), (dict(M=0, X=0), OK), (dict(N=0), OK),
    (dict(G=1024, N=1 << 21), UNS), (dict(N=1 << 25, K=1 << 20), UNS)])
def test_matvec4(L, kw, rc):
    p = dict(x=FAKE, dt=0, X=4, ids=FAKE, M=8, N=64, K=64, G=4, ep=_ep(), out=FAKE)
    p.update(kw)
    ep = ctypes.byref(p["ep"]) if p["ep"] is not None else None
    cfg = fos.Config().c(True)
    assert L.fos_matvec4(p["x"], p["dt"], p["X"], p["ids"], FAKE, FAKE, FAKE, p["M"], p["N"], p["K"], p["G"],
                         ctypes.byref(cfg), ep, p["out"], None) == rc


def test_matvec4_configurations(L):
    def call(cfg):
        ep = _ep()
        return L.fos_matvec4(FAKE, 0, 4, FAKE, FAKE, FAKE, FAKE, 8, 64, 64, 4, ctypes.byref(cfg) if cfg else None,
                             ctypes.byref(ep), FAKE, None)
    assert call(None) == INV and call(fos.Config(block16x16=True).c(True)) == UNS
    assert call(fos.Config(bound=44).c(True)) == UNS


def test_overlaps(L):
    """Outputs over inputs or one another; out over a part of the residual."""
    at = lambda n: ctypes.c_void_p(0x100000 + n)  # noqa: E731
    ep = _ep()
    far = [at(n << 20) for n in range(1, 8)]
    assert L.fos_linear8_grouped(far[0], far[1], far[2], far[3], far[4], 2, 16, 64, 128, ctypes.byref(ep),
                                 far[0], None) == INV
    ep = _ep(residual=far[5].value)
    assert L.fos_linear8_grouped(far[0], far[1], far[2], far[3], far[4], 2, 16, 64, 128, ctypes.byref(ep),
                                 ctypes.c_void_p(far[5].value + 128), None) == INV
    assert L.fos_quantize8_grouped(far[0], 0, 16, 64, far[1], 2, far[2], far[3], far[2], far[4], None) == INV
    assert L.fos_linear8_grouped_wgrad(far[0], far[1], far[2], far[3], far[4], 2, 16, 64, 64, None, 2, far[4],
                                       None) == INV
    ep = _ep()
    assert L.fos_matvec4(far[0], 0, 4, far[1], far[2], far[3], far[4], 8, 64, 64, 4,
                         ctypes.byref(fos.Config().c(True)), ctypes.byref(ep), far[3], None) == INV


def test_the_binding_wants_cuda_tensors():
    c, s = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    w, o = torch.zeros(2, 16, 128, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: fos.linear8_grouped(c, s, w, s, o), lambda: fos.quantize8_grouped(torch.zeros(4, 32), o),
                 lambda: fos.act_backward_grouped(torch.zeros(4, 32), None, "none", o),
                 lambda: fos.linear8_grouped_wgrad(c, s, c, s, o, 4),
                 lambda: fos.matvec4(torch.zeros(4, 32), c, s, torch.zeros(1))):
        with pytest.raises(ValueError):
            call()


def _text(name):
    with open(os.path.join(fos_build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_waits_for_the_other_cta_are_at_cluster_scope():
    """Barriers of fos_grouped.cuh that the other CTA of a pair arrives at, copies to or
    commits to are waited for at cluster scope (as test_pair_barriers_cpu.py has it)."""
    remote = {"full", "empty", "acc_full", "acc_empty", "sf_ready", "sf_free", "done"}
    seen = set()
    for kind, scope, bar in re.findall(r"(warp_wait|mbar_ask)(?:<Sync::(\w+)>)?\(&sh\.(\w+)", _text("fos_grouped.cuh")):
        if bar in remote:
            seen.add(bar)
            assert scope in ("CLUSTER", "TENSOR"), (kind, bar, scope)
        if bar == "full":
            assert scope == "CLUSTER", (kind, bar, scope)
    assert seen == remote


def test_kernels_wait_before_their_first_load():
    for name in ("fos_grouped.cuh", "fos_grouped_rows.cuh", "fos_matvec.cuh", "fos_quant8.cuh"):
        text = _text(name)
        assert "__ldg" not in text
        kernels = re.findall(r"__global__[^;{]*\)\s*\{(.*?)\n\}", text, flags=re.S)
        assert kernels
        for k in kernels:
            before = k.split("chain_wait();")[0]
            assert before != k
            assert not re.search(r"offs|ids\b.*a\.|a\.(x|ep|ts|scales|codes)\b|tma_load|pair_load", before), before
