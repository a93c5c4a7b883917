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


def _sweep(v, act, dt, rows):
    """The epilogue's activation at the values v (a multiple of 16 of them), as
    (outputs, pre-activations) of a product of zeros with v as the bias."""
    n = v.numel()
    a = fos.quantize8(torch.zeros(rows, 32, device=DEV))
    b = fos.quantize8(torch.zeros(n, 32, device=DEV))
    out, pre = fos.linear8(a[0], a[1], b[0], b[1], act=act, bias=v, out_dtype=dt, save_pre=True)
    bits = lambda t: t.view({4: torch.int32, 2: torch.int16}[t.element_size()])  # noqa: E731
    assert all(torch.equal(bits(t), bits(t[:1]).expand_as(t)) for t in (out, pre))
    return out[0], pre[0]


def _rel(act, v):
    """Relative error of the factor that the activation multiplies v by, where v < 0:
    silu       9 e: 2^x 4, its argument's remainder 1, the sum 1, the reciprocal 2,
               the product 1 (below -80: expf twice 4, two products 2)
    gelu_tanh  8 e, and the argument z = 2u of the exponential with 3.5 e |z|: two
               squares' and sums' roundings, two constants, the product
    gelu       the tail's polynomial: fit 1 e, evaluation 1 e and, per unit of |v|, 4.5 e at
               most (Horner's roundings, its argument with 4 e), of which no more than
               6.2 are granted; 2^x 4, products 2, the last rounding 1; the exponential's
               argument v^2 / 2 with 2.5 e of itself"""
    if act == "silu":
        return torch.full_like(v, 10 * E)
    if act == "gelu_tanh":
        return E * (9 + 3.5 * (2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)).abs())
    return E * (9 + (4.5 * v.abs()).clamp(max=6.2) + 1.25 * v * v)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("rows", [1, 3, 700])
def test_activation_relative_to_its_result(act, rows):
    """fp32 outputs over -100 .. 100 and out to the type's ends, from the kernel for
    few tokens and the one for many: the error is relative to the result, also
    in the negative tail, down to results of 2^-110."""
    lin = torch.linspace(-12, 12, 4096 * 3, device=DEV)
    wide = torch.linspace(-100, 100, 4096, device=DEV)
    far = torch.exp2(torch.linspace(-120, 127.9, 1024, device=DEV))
    v = torch.cat((lin, wide, far, -far))
    out, pre = _sweep(v, act, F32, rows)
    assert torch.equal(pre, v)
    v = v.to(D)
    want = _act64(v, act)
    if act == "relu":
        assert torch.equal(out.to(D), want)
        return
    r = _rel(act, v)
    neg = want.abs() * r
    # v > 0: v - |v| tail(v), or v times a factor of which 1 - s is off by what the
    # negative side's is, with the sum's, the reciprocal's and the product's roundings
    pos = want.abs() * 4 * E + (_act64(-v, act)).abs() * r
    bound = torch.where(v < 0, neg, pos) + 2.0 ** -110
    ref.near(out, want, bound, act)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_activation_of_16_bit_outputs(act, dt):
    """16-bit outputs over -80 .. 80: the type's rounding, and of the shorter forms silu's
    argument (1.5 e |v|: its rounding and the constant's) and gelu's tail (within 5.5e-6
    of itself to 3, 1.1e-4 to 6, 1.1e-3 to 9, 5e-3 beyond)."""
    v = torch.cat((torch.linspace(-12, 12, 4096 * 3, device=DEV), torch.linspace(-80, 80, 4096, device=DEV)))
    for rows in (1, 700):
        out, _ = _sweep(v, act, dt, rows)
        x = v.to(D)
        want = _act64(x, act)
        if act == "relu":
            r = torch.zeros_like(x)
        elif act == "silu":
            r = E * (10 + 1.5 * x.abs())
        else:
            r = _rel(act, x)
        if act == "gelu":
            a = x.abs()
            r = r + torch.where(a <= 3, 5.5e-6, torch.where(a <= 6, 1.1e-4, torch.where(a <= 9, 1.1e-3, 5e-3)))
        bound = torch.where(x < 0, want.abs() * r, want.abs() * 4 * E + _act64(-x, act).abs() * r)
        ref.near(out, want, bound * 1.01 + want.abs() * ref.U[dt] * (1 + 2.0 ** -7) + ref.TINY[dt] + 2.0 ** -117, act)


def test_silu_below_the_range_of_the_exponential():
    """silu down to -103, where exp(-v) leaves fp32's range at -88.7 and the result
    itself only below -92: relative to the result, to a subnormal's spacing."""
    v = torch.linspace(-103.9, -70, 4096, device=DEV)
    for rows in (1, 700):
        out, _ = _sweep(v, "silu", F32, rows)
        want = _act64(v.to(D), "silu")
        ref.near(out, want, want.abs() * 10 * E + 2.0 ** -149, "silu")


def test_activations_of_infinities_and_nan():
    """As the formulas give them: inf, and inf * 0 = NaN on the negative side."""
    v = torch.tensor([math.inf, -math.inf, math.nan, 1.0] * 4, device=DEV)
    for rows in (1, 700):
        for act in ("relu", "gelu", "gelu_tanh", "silu"):
            out, _ = _sweep(v, act, F32, rows)
            assert out[0].item() == math.inf and math.isnan(out[2].item())
            assert out[1].item() == 0 if act == "relu" else math.isnan(out[1].item())
            assert math.isfinite(out[3].item())


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_derivative_relative_to_its_terms(act):
    """act_backward in fp32 with dout = 1 over -30 .. 30: the error is relative to
    the sizes of the derivative's terms, which vanish in the negative tail.
      gelu       Phi + p phi: Phi's tail as in _rel, phi with 4 e (2^x), 2.5 e of its
                 argument and 3 e of products; the sum's rounding
      the others s + p z' s (1 - s) with s of relative error r = 9 e + 3.5 e |z|
                 (silu z = p: 1.5 e |z|): r s (1 - s) from the exponential and 3 e s from the
                 rest in each s, 1 - s with e more, products 4 e"""
    p = torch.cat((torch.linspace(-12, 12, 16384, device=DEV), torch.linspace(-30, 30, 4096, device=DEV)))
    d = fos.act_backward(torch.ones(64, 320, device=DEV), p.view(64, 320).contiguous(), act,
                         rowwise=False, colwise=False, value=True, bias_grad=False)[4].view(-1)
    p = p.to(D)
    want = _slope64(p, act)
    if act == "gelu":
        phi = torch.exp(-p * p / 2) / math.sqrt(2 * math.pi)
        tail = 0.5 * torch.erfc(p.abs() / math.sqrt(2))
        bound = (tail * E * (15.2 + 1.25 * p * p) + (p > 0) * E
                 + p.abs() * phi * E * (7.5 + 1.25 * p * p) + want.abs() * E)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        z, dz = (p, 1) if act == "silu" else (c * (p + 0.044715 * p ** 3), c * (1 + 0.134145 * p * p))
        s, r = torch.sigmoid(z), torch.sigmoid(-z)
        es = s * r * E * (4 + (1.5 if act == "silu" else 3.5) * z.abs()) + s * 3 * E
        bound = es + (p * dz).abs() * (es * r + s * (es + r * E) + s * r * 4 * E) + want.abs() * 2 * E
    ref.near(d, want, bound * 1.02 + 2.0 ** -110, act)


@pytest.mark.parametrize("act,lo,hi,limit", [
    ("gelu", -1, 0, 0.4), ("gelu", 0, 1, 0.6), ("gelu", 1, 6, 0.8), ("gelu_tanh", -1, 0, 0.6),
    ("gelu_tanh", 0, 1, 1.0), ("gelu_tanh", 1, 6, 1.5)])
def test_derivative_root_mean_square(act, lo, hi, limit):
    """Where most pre-activations are, the root mean square error in units of e: a
    rounding of a value of 1/2 .. 1 is 0.29 (0.58 from 1 up), the last one and, of
    gelu, one of q and the exponential's, of gelu_tanh a few more in s and in
    p z' s (1 - s), whose size is at most 0.6; no cancellation adds to them."""
    p = torch.linspace(lo, hi, 1 << 18, device=DEV)
    d = fos.act_backward(torch.ones(512, 512, device=DEV), p.view(512, 512), act, rowwise=False,
                         colwise=False, value=True, bias_grad=False)[4].view(-1)
    off = ((d.to(D) - _slope64(p.to(D), act)) ** 2).mean().sqrt().item() / E
    assert off < limit, off


@pytest.mark.parametrize("cols", [32 * 49, 32 * 41, 2080, 7168, 7456, 8224, 14336, 16416])
def test_rstd_has_no_bias(cols):
    """Rows of small integers, whose sums of squares are exact: what is left in rstd
    are roundings of either sign, at most 2 e in each row, so their mean over n
    rows is within 5 * 2 e / sqrt(3 n) (five standard deviations of uniform errors),
    for widths that are no power of two as well.  1 / cols rounded to fp32 has one
    error in every row."""
    g = torch.Generator(device=DEV)
    g.manual_seed(cols)
    n = 20000
    x = torch.randint(-3, 4, (n, cols), generator=g, device=DEV).to(BF16)
    x[:, 0] = 1
    rstd = fos.rms_norm(x, torch.ones(cols, device=DEV), eps=0.0, quantized=False)[4]
    want = 1 / x.float().square().sum(1).to(D).div(cols).sqrt()
    off = rstd.to(D) / want - 1
    assert off.abs().max() < 2 * E
    assert abs(off.mean().item()) < 10 * E / math.sqrt(3 * n), off.mean().item() / E


def _rand(rows, cols, dt, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(rows, cols, generator=g, device=DEV).to(dt)


@pytest.mark.parametrize("cols", [64, 2048, 4096, 16384, 16416])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_norm_in_place(cols, dt):
    """h in the place of the residual or of x."""
    for rows in (1, 700):
        x, r, w = _rand(rows, cols, dt, 1), _rand(rows, cols, dt, 2), torch.ones(cols, device=DEV)
        want = fos.rms_norm(x, w, r, normalized=True)
        for which in (0, 1):
            a, b = x.clone(), r.clone()
            got = fos.rms_norm(a, w, b, normalized=True, h=(a, b)[which])
            assert got[3] is (a, b)[which]
            assert all(torch.equal(p, q) for p, q in zip(got, want))
            assert torch.equal((a, b)[1 - which], (x, r)[1 - which])


@pytest.mark.parametrize("cols", [64, 4096, 8192, 8224])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_norm_backward_in_place(cols, dt):
    """dx in the place of dy, h or dh."""
    for rows in (1, 700):
        dy, h, dh = (_rand(rows, cols, dt, k) for k in (1, 2, 3))
        rstd, w = torch.rand(rows, device=DEV) + 0.5, torch.rand(cols, device=DEV) + 0.5
        want = fos.rms_norm_backward(dy, h, rstd, w, dh)
        for which in range(3):
            t = [dy.clone(), h.clone(), dh.clone()]
            got = fos.rms_norm_backward(t[0], t[1], rstd, w, t[2], dx=t[which])
            assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_act_backward_in_place():
    """d in the place of dout or of pre."""
    for dt in (BF16, F32):
        dout, pre = _rand(517, 1088, dt, 1), _rand(517, 1088, dt, 2)
        want = fos.act_backward(dout, pre, "silu", value=True)
        for which in (0, 1):
            t = [dout.clone(), pre.clone()]
            got = fos.act_backward(*t, "silu", value=True, d=t[which])
            assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("fmt", [8, 4])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_linear_in_place(fmt, dt):
    """out in the place of the residual: a residual stream updated where it is."""
    for M, N, K in ((1, 16, 64), (5, 16, 64), (48, 4096, 1024), (300, 48, 4096), (1500, 2064, 256)):
        a, b, r = _rand(M, K, BF16, 1), _rand(N, K, BF16, 2), _rand(M, N, dt, 3)
        if fmt == 8:
            (ac, as_, _, _), (bc, bs, _, _) = fos.quantize8(a), fos.quantize8(b)
            call = lambda res, **kw: fos.linear8(ac, as_, bc, bs, residual=res, out_dtype=dt, **kw)  # noqa: E731
        else:
            cfg = fos.Config(scale_tiled=True)
            qa, qb = fos.quantize(a, cfg), fos.quantize(b, cfg)
            call = lambda res, **kw: fos.linear4(*qa, *qb, residual=res, out_dtype=dt, **kw)  # noqa: E731
        want, t = call(r), r.clone()
        assert call(t, out=t) is t and torch.equal(t, want)


def test_overlaps_are_refused():
    """An output may be the same tensor as the inputs named in the header; any
    other overlap is refused before a launch."""
    buf = torch.zeros(4 * 64 * 64, dtype=BF16, device=DEV)
    at = lambda o, r=64, c=64: buf[o:o + r * c].view(r, c)  # noqa: E731
    x, res, w = at(0), at(4096), torch.ones(64, device=DEV)
    rstd = torch.ones(64, device=DEV)
    u8 = buf.view(torch.uint8)
    bad = [
        lambda: fos.rms_norm(x, w, res, h=at(64)),
        lambda: fos.rms_norm(x, w, res, h=at(4096 - 64)),
        lambda: fos.rms_norm(x, w, normalized=True, y=x),
        lambda: fos.rms_norm(x, w, res, normalized=True, y=at(12288), h=at(12288)),
        lambda: fos.rms_norm(x, w, codes=u8[:4096].view(64, 64)),
        lambda: fos.rms_norm_backward(x, res, rstd, w, dx=at(4096 + 64)),
        lambda: fos.rms_norm_backward(x, res, rstd, w, dweight=rstd),
        lambda: fos.act_backward(x, res, "silu", value=True, d=at(64)),
        lambda: fos.quantize8(x, codes=u8[:4096].view(64, 64)),
        lambda: fos.act_backward(at(0, 256), at(0, 256), "silu", dbias=buf.view(F32)[:64]),
    ]
    for f in bad:
        with pytest.raises(fos.FosError) as e:
            f()
        assert e.value.status == fos.FOS_ERR_INVALID_ARG
    ac, as_, _, _ = fos.quantize8(x)
    r2 = at(4096)
    for kw in (dict(residual=r2, out=at(4096 + 64)), dict(out=at(0), pre=at(0), save_pre=True),
               dict(residual=r2, pre=r2, save_pre=True), dict(bias=r2[0], out=r2)):
        with pytest.raises(fos.FosError) as e:
            fos.linear8(ac, as_, ac, as_, **kw)
        assert e.value.status == fos.FOS_ERR_INVALID_ARG


def test_kept_workspaces_are_bounded_and_released():
    """A thread keeps the workspaces of the streams that it used last, at most
    eight, and gives them back when asked."""
    dy, h = _rand(300, 512, BF16, 1), _rand(300, 512, BF16, 2)
    rstd, w = torch.ones(300, device=DEV), torch.ones(512, device=DEV)
    want = fos.rms_norm_backward(dy, h, rstd, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(12)]
    for s in streams + streams[:3]:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = fos.rms_norm_backward(dy, h, rstd, w)
        s.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert len(fos._kept.__dict__) <= 8
        assert list(fos._kept.__dict__)[-1] == (dy.get_device(), s.cuda_stream)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    held = sum(v.numel() for v in fos._kept.__dict__.values())
    fos.release_workspaces()
    assert not fos._kept.__dict__ and before - torch.cuda.memory_allocated() >= held > 0
    got = fos.rms_norm_backward(dy, h, rstd, w)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
