"""Feed-forward operators where their arithmetic can go wrong: activations and
their derivatives over the whole range of fp32 with bounds relative to the
result, rows whose statistics are exact, rows of tiny values without eps,
outputs that take the place of an input.

e = 2^-24.  Errors of what the kernels use, from the PTX and CUDA documents:
2^x 4e (ex2.approx), the reciprocal 2e (rcp.approx), expf 2e; a rounding e; a
constant e / 2.
"""
import math

import pytest
import torch

import ffn_reference as ref
import nvfp4_quantization_precision_gb300 as fos

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = torch.float64
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E = 2.0 ** -24
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _act64(v, name):
    """The activation without cancellation on the negative side."""
    if name == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return ref.act(v, name)


def _slope64(p, name):
    """The derivative, each term formed so that a zero factor wins over the
    other's size."""
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        q = p.clamp(-40, 40)
        s, r = (torch.sigmoid(k * c * (q + 0.044715 * q ** 3)) for k in (1, -1))
        return s + q * c * (1 + 3 * 0.044715 * q * q) * s * r
    if name == "silu":
        q = p.clamp(-1000, 1000)
        return torch.sigmoid(q) + q * torch.sigmoid(q) * torch.sigmoid(-q)
    return ref.act_slope(p, name)


LARGE = [1e2, 1e4, 3e4, 65504.0, 1.1e13, 1.2e13, 1.3e13, 1e14, 1e19, 2e19, 1e30, 3.38e38]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_act_backward_of_large_values(act, dt):
    """Large finite pre-activations: the derivative is 0 or 1 there, to the bit,
    in d, both quantized forms and the bias gradient."""
    vals = [v for v in LARGE if v <= torch.finfo(dt).max]
    rows = 2 * len(vals)
    p = torch.tensor(vals + [-v for v in vals], device=DEV).to(dt).view(-1, 1).repeat(1, 64)
    dout = torch.full((rows, 64), 0.5, dtype=dt, device=DEV)
    codes, scales, codes_t, scales_t, d, db = fos.act_backward(
        dout, None if act == "none" else p, act, scale_tiled=False, value=True)
    want = torch.full((rows, 64), 0.5, dtype=D)
    if act != "none":
        want[len(vals):] = 0
    assert torch.equal(d.to(D).cpu(), want)
    assert torch.equal(db.to(D).cpu(), want.sum(0))
    q, s = ref.quantize8(want)
    assert torch.equal(ref.e4m3(codes), q) and torch.equal(scales.cpu().long(), s)
    pad = torch.zeros(64, codes_t.shape[1], dtype=D)
    pad[:, :rows] = want.t()
    q, s = ref.quantize8(pad)
    assert torch.equal(ref.e4m3(codes_t), q) and torch.equal(scales_t.cpu().long(), s)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_act_backward_of_infinities_and_nan(act, dt):
    """An infinite or NaN pre-activation leaves NaN (relu: 1 or 0, and 0) in its
    own element and nothing elsewhere."""
    p = torch.full((40, 96), 0.5, dtype=dt, device=DEV)
    at = {(3, 5): math.inf, (7, 40): -math.inf, (35, 70): math.nan}
    for (r, c), v in at.items():
        p[r, c] = v
    dout = torch.ones_like(p)
    codes, _, codes_t, _, d, db = fos.act_backward(dout, None if act == "none" else p, act,
                                                   scale_tiled=False, value=True)
    d = d.to(D).cpu()
    if act == "none":
        assert (d == 1).all()
        return
    got = {k: d[k].item() for k in at}
    if act == "relu":
        assert got == {(3, 5): 1.0, (7, 40): 0.0, (35, 70): 0.0}
    else:
        assert all(math.isnan(v) for v in got.values())
        assert int(torch.isnan(ref.e4m3(codes)).sum()) == 3
        assert int(torch.isnan(ref.e4m3(codes_t)).sum()) == 3
        assert int(torch.isnan(db).sum()) == 3
    for k in at:
        d[k] = d[0, 0]
    assert (d == d[0, 0]).all() and torch.isfinite(d).all()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("cols", [64, 1024, 4096, 8192, 8224, 16416])
def test_rms_norm_backward_of_tiny_rows(cols, dt):
    """Rows of about 1e-20 and 1e-21 with the rstd that eps = 0 gives them (up to
    1e21), gradients of ordinary and of small size: dx is in range, and so is
    every step to it.  Bounds as for ordinary rows: e per rounding and per unit
    of the terms' sizes, the sum's error 40 e (a chain of 16 terms and a tree)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(cols)
    rows = 24
    size = torch.tensor([1e-20, 1e-21, 1.0], device=DEV).repeat(8).unsqueeze(1)
    h = (torch.randn(rows, cols, generator=g, device=DEV) * size).to(dt)
    rstd = (1 / h.to(D).square().mean(1).sqrt()).float()
    up = torch.tensor([1.0, 1e-3, 1e-18], device=DEV).repeat_interleave(8).unsqueeze(1)
    dy = (torch.randn(rows, cols, generator=g, device=DEV) * up).to(dt)
    w = 1 + 0.1 * torch.randn(cols, generator=g, device=DEV)
    for dh in (None, dy.flip(0).contiguous()):
        dx, dw = fos.rms_norm_backward(dy, h, rstd, w, dh)
        gr, xh, r = dy.to(D) * w.to(D), h.to(D) * rstd.to(D).unsqueeze(1), rstd.to(D).unsqueeze(1)
        want = r * (gr - xh * (gr * xh).mean(1, keepdim=True)) + (dh.to(D) if dh is not None else 0)
        size = r * (gr.abs() + xh.abs() * (gr * xh).abs().mean(1, keepdim=True) * 40)
        bound = want.abs() * ref.U[dt] + (size + want.abs()) * 8 * E + ref.TINY[dt]
        ref.near(dx, want, bound, "dx")
        t = dy.to(D) * xh
        ref.near(dw, t.sum(0), t.abs().sum(0) * (rows + 8) * E, "dweight")
