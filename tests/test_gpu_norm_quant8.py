"""The norm, its backward pass and the 8-bit quantization against plain 64-bit
forms (ffn_reference), over types, widths that take every launch variant,
ragged row counts, both scale layouts and special values; repeat calls bit
for bit; refusals.

Bounds (u = unit roundoff of the stored type, e = 2^-24 of fp32):
  rstd   relative 2^-22: the sum of squares in fp32 (per-thread chains of at
         most 16 terms and a tree, gamma_16 e = 2^-20 worst case, random in
         sign; 2^-22 is a quarter of that)
  y      relative 2^-21 before its rounding: rstd's bound and three roundings
  dx     u |dx| + 2^-21 (|g rstd| + |h c| + |dh|) + the sum's error: at most
         C e per unit of sum |g h|, rstd^3 |h| / C times that
  dw     gamma_n sum |dy h rstd|, n = rows + 8 (a chain per CTA, a tree after)
  slope  2^-19 absolute (at most |p| (1 - s) with an absolute error of e for
         |p| < 17, exp and erf within 2 ulp)
"""
import ctypes
import threading

import pytest
import torch

import ffn_reference as ref
import nvfp4_quantization_precision_gb300 as fos

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = torch.float64
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _rand(rows, cols, dt, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device=DEV) * scale
    x = torch.where(torch.rand(rows, cols, generator=g, device=DEV) < 2e-3, x * 30, x)
    return x.to(dt)


def _filled(shape):
    return torch.full(shape, 0xFF, dtype=torch.uint8, device=DEV)


def _plain_scales(scales, rows, n, tiled):
    if not tiled:
        return scales.view(rows, n)
    assert (ref.padding(scales, rows, n) == 0).all(), "padding of the tiled scales"
    return ref.untile(scales, rows, n)


def _check_norm(x, w, r, eps, tiled, out):
    codes, scales, y, h, rstd = out
    R, C = x.shape
    h64 = x.to(D) + (r.to(D) if r is not None else 0)
    rs = 1 / torch.sqrt((h64 * h64).mean(1) + eps)
    ref.near(rstd, rs, rs * 2.0 ** -22, "rstd")
    if r is not None:
        ref.near(h, h64, h64.abs() * (ref.U[x.dtype] + 2.0 ** -23) + ref.TINY[x.dtype], "h")
    y64 = h64 * rs.unsqueeze(1) * w.to(D)
    if codes is not None:
        ref.check_codes(codes, _plain_scales(scales, R, C // 32, tiled), y64, 2.0 ** -21)
    if y is not None:
        ref.near(y, y64, y64.abs() * (ref.U[x.dtype] + 2.0 ** -21) + ref.TINY[x.dtype], "y")


# widths: one warp with one and two segments a lane, 128 and 256 threads, two
# segments of 256 and 512 threads, and the two-sweep rows
WIDTHS = [32, 96, 512, 544, 1024, 2048, 2080, 4096, 4128, 8192, 8224, 16384, 16416, 20480]


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_rms_norm_widths(cols, dt):
    for rows, res, tiled, w32 in ((1, True, True, True), (5, False, False, False),
                                  (131, True, False, True), (33, False, True, True)):
        x, w = _rand(rows, cols, dt, cols + rows), _rand(1, cols, F32, 7)[0] * 0.1 + 1
        if not w32:
            w = w.to(dt)
        r = _rand(rows, cols, dt, 3, 2.0) if res else None
        n = fos.scales8_shape(rows, cols, tiled)
        out = fos.rms_norm(x, w, r, eps=1e-5, scale_tiled=tiled, normalized=True,
                           codes=_filled((rows, cols)), scales=_filled(n))
        _check_norm(x, w, r, 1e-5, tiled, out)


@pytest.mark.parametrize("rows", [2, 127, 128, 129, 700, 3001])
def test_rms_norm_rows(rows):
    x, w, r = _rand(rows, 1056, BF16, rows), _rand(1, 1056, BF16, 1)[0], _rand(rows, 1056, BF16, 2)
    _check_norm(x, w, r, 1e-6, True, fos.rms_norm(x, w, r, scales=_filled(
        fos.scales8_shape(rows, 1056))))


def test_rms_norm_many_rows_of_every_group():
    """More rows than the grid holds at once: the loop over rows with its next
    row in flight, in every launch variant."""
    for cols in (64, 1024, 2048, 4096, 8192):
        x, w = _rand(6001, cols, BF16, cols), torch.ones(cols, device=DEV)
        _check_norm(x, w, None, 1e-6, True, fos.rms_norm(x, w))


def test_rms_norm_only_what_is_asked_for():
    x, w = _rand(9, 256, BF16, 1), torch.ones(256, device=DEV)
    codes, scales, y, h, rstd = fos.rms_norm(x, w)
    assert y is None and h is x
    c2, s2, y2, _, r2 = fos.rms_norm(x, w, quantized=False, normalized=True)
    assert c2 is None and s2 is None and torch.equal(rstd, r2)
    _check_norm(x, w, None, 1e-6, True, (None, None, y2, None, r2))


def test_rms_norm_special_rows():
    """All-zero rows, an infinity, a NaN, subnormals, rows whose squares
    overflow or underflow fp32."""
    C = 512
    for dt in (BF16, F32):
        x = _rand(8, C, dt, 1)
        x[0] = 0
        x[1, 5] = float("inf")
        x[2, 40] = float("nan")
        x[3] = 1e-39 if dt == F32 else 1e-38
        x[4] = 3e19
        x[5] = 1e-22
        x[6, 64:] = 0
        w = torch.ones(C, device=DEV)
        codes, scales, y, h, rstd = fos.rms_norm(x, w, scale_tiled=False, normalized=True)
        got = ref.e4m3(codes)
        assert rstd[0].item() == pytest.approx(1e3, rel=1e-6) and (codes[0] == 0).all()
        assert (scales[0] == 0).all()
        assert rstd[1].item() == 0 and torch.isnan(got[1, 5]) and (got[1, :5] == 0).all()
        assert torch.isnan(rstd[2]) and torch.isnan(got[2]).all() and (scales[2] == 0).all()
        assert rstd[4].item() == 0 and (got[4] == 0).all()
        assert torch.isfinite(got[3]).all() and torch.isfinite(got[5:]).all()
        keep = [0, 3, 5, 6, 7]
        _check_norm(x[keep], w, None, 1e-6, False, (codes[keep], scales[keep].contiguous(), None,
                                                    None, rstd[keep]))


def test_rms_norm_two_calls_one_answer():
    x, w, r = _rand(300, 4096, BF16, 5), torch.ones(4096, device=DEV), _rand(300, 4096, BF16, 6)
    a, b = fos.rms_norm(x, w, r), fos.rms_norm(x, w, r)
    for p, q in zip(a, b):
        assert (p is None and q is None) or torch.equal(p, q)


@pytest.mark.parametrize("cols", [32, 480, 512, 544, 1024, 2048, 4096, 4128, 8192, 8224, 16416])
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_rms_norm_backward(cols, dt):
    for rows, use_dh, w32 in ((1, True, True), (7, False, False), (150, True, True),
                              (1003 if cols <= 2048 else 401, False, True)):
        h = _rand(rows, cols, dt, rows + cols)
        rstd = (1 / torch.sqrt(h.to(D).square().mean(1) + 1e-6)).float()
        dy, dh = _rand(rows, cols, dt, 2, 0.1), _rand(rows, cols, dt, 3, 0.1) if use_dh else None
        w = _rand(1, cols, F32, 4)[0] * 0.2 + 1
        if not w32:
            w = w.to(dt)
        dx, dw = fos.rms_norm_backward(dy, h, rstd, w, dh)
        h6, g, r = h.to(D), dy.to(D) * w.to(D), rstd.to(D).unsqueeze(1)
        c = r ** 3 * (g * h6).mean(1, keepdim=True)
        want = r * g - h6 * c + (dh.to(D) if use_dh else 0)
        s_err = r ** 3 * (g * h6).abs().sum(1, keepdim=True) * 2.0 ** -24
        bound = (want.abs() * ref.U[dt] + 2.0 ** -21 * ((r * g).abs() + (h6 * c).abs() + want.abs())
                 + h6.abs() * s_err + ref.TINY[dt])
        ref.near(dx, want, bound, "dx")
        t = dy.to(D) * h6 * r
        ref.near(dw, t.sum(0), t.abs().sum(0) * (rows + 8) * 2.0 ** -24 + 1e-30, "dweight")
        dx2, none = fos.rms_norm_backward(dy, h, rstd, w, dh, weight_grad=False)
        assert none is None and torch.equal(dx, dx2)


def test_rms_norm_backward_against_differences():
    """Central differences of a scalar of the forward pass (fp32 output y,
    64-bit sums): the step 2^-7 leaves the cubic term, about h^2 = 6e-5 of the
    gradient's size, and y's rounding 2^-24 / step, so 1e-3 bounds both."""
    R, C = 3, 64
    x, r = _rand(R, C, F32, 1), _rand(R, C, F32, 2)
    w, dy = _rand(1, C, F32, 3)[0] * 0.1 + 1, _rand(R, C, F32, 4)
    gen = torch.Generator().manual_seed(0)

    def f(xx, ww):
        y = fos.rms_norm(xx, ww, r, quantized=False, normalized=True)[2]
        return (y.to(D) * dy.to(D)).sum().item()

    _, _, _, h, rstd = fos.rms_norm(x, w, r, quantized=False)
    dx, dw = fos.rms_norm_backward(dy, h, rstd, w)
    step = 2.0 ** -7
    for _ in range(40):
        i, j = int(torch.randint(R, (1,), generator=gen)), int(torch.randint(C, (1,), generator=gen))
        e = torch.zeros_like(x)
        e[i, j] = step
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * step) - dx[i, j].item()) < 1e-3 * max(
            1.0, dx.abs().max().item())
        ew = torch.zeros_like(w)
        ew[j] = step
        assert abs((f(x, w + ew) - f(x, w - ew)) / (2 * step) - dw[j].item()) < 1e-3 * max(
            1.0, dw.abs().max().item())


# ------------------------------------------------------------------ quantize8
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (32, 128), (33, 160), (127, 96), (128, 256),
                                       (129, 288), (300, 1056), (1000, 2048)])
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_quantize8_is_exact(rows, cols, dt):
    """Quantization alone has one rounding: codes and scales equal the exact ones."""
    x = _rand(rows, cols, dt, rows * 7 + cols, 0.3)
    x[0, :8] = 0
    x[-1, 32 * (cols // 64):32 * (cols // 64) + 32] = 0
    pad = -(-rows // 32) * 32
    xt = torch.zeros(cols, pad, dtype=D)
    xt[:, :rows] = x.to(D).cpu().t()
    for tiled in (True, False):
        n, nt = fos.scales8_shape(rows, cols, tiled), fos.scales8_shape(cols, pad, tiled)
        got = fos.quantize8(x, scale_tiled=tiled, colwise=True, codes=_filled((rows, cols)),
                            scales=_filled(n), codes_t=_filled((cols, pad)), scales_t=_filled(nt))
        for v, c, s, R, N in ((x.to(D).cpu(), got[0], got[1], rows, cols // 32),
                              (xt, got[2], got[3], cols, pad // 32)):
            q, sc = ref.quantize8(v)
            assert torch.equal(_plain_scales(s, R, N, tiled).cpu().long(), sc)
            assert torch.equal(ref.e4m3(c), q)
        rows_only = fos.quantize8(x, scale_tiled=tiled)
        cols_only = fos.quantize8(x, scale_tiled=tiled, rowwise=False, colwise=True)
        assert torch.equal(rows_only[0], got[0]) and torch.equal(rows_only[1], got[1])
        assert torch.equal(cols_only[2], got[2]) and torch.equal(cols_only[3], got[3])
        assert rows_only[2] is None and cols_only[0] is None


def test_quantize8_thresholds_and_specials():
    """Amaxes on and next to the 448 * 2^e thresholds, the ends of the fp32
    range, infinities and NaN."""
    vals = []
    for e in (-126, -20, 0, 5, 100):
        for m in (1.0, 1.75, 1.75 * (1 - 2.0 ** -23), 1.75 * (1 + 2.0 ** -23), 1.999):
            vals.append(m * 2.0 ** e)
    vals += [0.0, 2.0 ** -149, 448.0, 449.0, 3.4e38, float("inf"), float("nan")]
    x = torch.zeros(len(vals), 64, device=DEV)
    for i, v in enumerate(vals):
        x[i, 3] = v
        x[i, 9] = -v / 3
        x[i, 40] = v / 1e3
    got = fos.quantize8(x, scale_tiled=False)
    q, sc = ref.quantize8(x.to(D).cpu())
    assert torch.equal(got[1].cpu().long(), sc)
    g = ref.e4m3(got[0])
    assert torch.equal(torch.isnan(g), torch.isnan(q))
    assert torch.equal(torch.nan_to_num(g), torch.nan_to_num(q))


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_act_backward(act, dt):
    for rows, cols in ((1, 32), (65, 224), (128, 128), (517, 1088)):
        dout, pre = _rand(rows, cols, dt, rows, 0.1), _rand(rows, cols, dt, cols, 1.5)
        pre[0, :3] = 0
        d64 = dout.to(D) * ref.act_slope(pre.to(D), act)
        err = dout.to(D).abs() * (0 if act in ("none", "relu") else 2.0 ** -19)
        pad = -(-rows // 32) * 32
        tiled = rows != 65
        codes, scales, codes_t, scales_t, d, dbias = fos.act_backward(
            dout, None if act == "none" else pre, act, scale_tiled=tiled, value=True)
        ref.near(d, d64, err + d64.abs() * (ref.U[dt] + 2.0 ** -23) + ref.TINY[dt], "d")
        rel = torch.where(d64 != 0, err / d64.abs().clamp(min=1e-300) + 2.0 ** -23, 0 * d64)
        # an element's bound in its block's units: the largest absolute one
        _codes(codes, _plain_scales(scales, rows, cols // 32, tiled), d64.cpu(), err.cpu())
        t, te = torch.zeros(cols, pad, dtype=D), torch.zeros(cols, pad, dtype=D)
        t[:, :rows], te[:, :rows] = d64.cpu().t(), err.cpu().t()
        _codes(codes_t, _plain_scales(scales_t, cols, pad // 32, tiled), t, te)
        ref.near(dbias, d64.sum(0), d64.abs().sum(0) * (rows + 8) * 2.0 ** -24 + err.sum(0) + 1e-30,
                 "dbias")
        del rel


def _codes(codes, scales, v, err):
    """check_codes with an absolute error per element."""
    s = scales.cpu().long()
    a, e = ref.amax_of(v), ref.amax_of(err)
    tol = e + a * 2.0 ** -23
    assert ((s >= ref.scale_of((a - tol).clamp(min=0))) & (s <= ref.scale_of(a + tol))).all()
    up = ref.pow2(127 - s).unsqueeze(2)
    y, got = ref.blocks(v) * up, ref.blocks(ref.e4m3(codes))
    _, k = torch.frexp(y.abs() + ref.blocks(err) * up)
    half = ref.pow2((k - 5).clamp(min=-10))
    off = (got - y.clamp(-448, 448)).abs()
    lim = half * (1 + 1e-12) + (ref.blocks(err) + ref.blocks(v).abs() * 2.0 ** -23) * up
    assert not (off > lim).any()


def test_act_backward_is_the_derivative_of_the_forward():
    """act_slope's closed forms against central differences of act (64 bits,
    step 1e-5: cubic term 1e-10, rounding 1e-11)."""
    p = torch.linspace(-6, 6, 1001, dtype=D) + 1e-3
    for a in ("relu", "gelu", "gelu_tanh", "silu"):
        num = (ref.act(p + 1e-5, a) - ref.act(p - 1e-5, a)) / 2e-5
        assert (num - ref.act_slope(p, a)).abs().max() < 1e-8


def test_act_backward_parts_agree():
    """Each output is the same whatever else is asked for; repeats are equal."""
    dout, pre = _rand(300, 416, BF16, 1), _rand(300, 416, BF16, 2)
    full = fos.act_backward(dout, pre, "silu", value=True)
    again = fos.act_backward(dout, pre, "silu", value=True)
    for p, q in zip(full, again):
        assert torch.equal(p, q)
    for k in ("rowwise", "colwise", "value", "bias_grad"):
        kw = dict(rowwise=False, colwise=False, value=False, bias_grad=False)
        kw[k] = True
        one = fos.act_backward(dout, pre, "silu", **kw)
        for p, q in zip(one, full):
            assert p is None or torch.equal(p, q)


def test_empty_rows():
    x = torch.empty(0, 256, dtype=BF16, device=DEV)
    w = torch.ones(256, device=DEV)
    codes, scales, _, _, rstd = fos.rms_norm(x, w)
    assert codes.shape == (0, 256) and scales.numel() == 0 and rstd.numel() == 0
    dx, dw = fos.rms_norm_backward(x, x, rstd, w)
    assert dx.shape == (0, 256) and (dw == 0).all()
    q = fos.quantize8(x, colwise=True)
    assert q[2].shape == (256, 0)
    assert (fos.act_backward(x, x, "gelu")[5] == 0).all()


def test_side_stream():
    """The calls run on the current stream, which need not be the tensors' own."""
    x, w = _rand(513, 2048, BF16, 1), torch.ones(2048, device=DEV)
    torch.cuda.synchronize()
    want, wq = fos.rms_norm(x, w), fos.act_backward(x, x, "gelu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got, gq = fos.rms_norm(x, w), fos.act_backward(x, x, "gelu")
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(gq[2], wq[2]) and torch.equal(gq[5], wq[5])


def test_graph_capture():
    x, w, r = (_rand(64, 1024, BF16, 1), torch.ones(1024, device=DEV), _rand(64, 1024, BF16, 2))
    want = [t.clone() for t in fos.rms_norm(x, w, r) if t is not None]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fos.rms_norm(x, w, r)
    for t in out:
        if t is not None:
            t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for p, q in zip([t for t in out if t is not None], want):
        assert torch.equal(p, q)


def test_kept_workspaces():
    """Calls without a workspace: any order of sizes gives what a workspace of
    the caller's gives; streams, threads and captured graphs do not share one."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(9)
    args = []
    for rows, cols in ((300, 512), (2000, 4096), (130, 64), (2000, 4096)):
        dy, h = (torch.randn(rows, cols, generator=gen, device=DEV).to(BF16) for _ in range(2))
        args.append((dy, h, torch.rand(rows, generator=gen, device=DEV) + 0.5,
                     torch.randn(cols, generator=gen, device=DEV)))
    give = [torch.empty(64 << 20, dtype=torch.uint8, device=DEV) for _ in args]

    def calls(ws):
        out = []
        for (dy, h, rstd, w), x in zip(args, ws):
            out += fos.rms_norm_backward(dy, h, rstd, w, workspace=x)
            out.append(fos.act_backward(dy, h, "silu", rowwise=False, colwise=False, workspace=x)[5])
        return out

    want = calls(give)
    none = [None] * len(args)
    assert all(torch.equal(p, q) for p, q in zip(calls(none), want))
    mine = dict(fos._kept.__dict__)
    assert len({v.data_ptr() for v in mine.values()}) == len(mine) and max(
        v.numel() for v in mine.values()) <= 16 << 20
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = {}
    with torch.cuda.stream(side):
        got["stream"] = calls(none)

    def other():
        got["thread"] = calls(none)
        got["kept"] = {v.data_ptr() for v in fos._kept.__dict__.values()}

    th = threading.Thread(target=other)
    th.start()
    got["main"] = calls(none)
    th.join()
    both = {v.data_ptr() for v in fos._kept.__dict__.values()}
    assert len(both) > len(mine) and not both & got["kept"]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got["graph"] = calls(none)
    assert {v.data_ptr() for v in fos._kept.__dict__.values()} == both
    g.replay()
    torch.cuda.synchronize()
    for k in ("stream", "thread", "main", "graph"):
        assert all(torch.equal(p, q) for p, q in zip(got[k], want)), k


def test_refusals():
    x, w = _rand(8, 64, BF16, 1), torch.ones(64, device=DEV)
    rstd = torch.ones(8, device=DEV)
    with pytest.raises(ValueError):
        fos.rms_norm(x.cpu(), w)
    with pytest.raises(ValueError):
        fos.rms_norm(x.t(), w)
    with pytest.raises(ValueError):
        fos.rms_norm(x, w.half())
    with pytest.raises(ValueError):
        fos.rms_norm(x, w, residual=x.float())
    with pytest.raises(ValueError):
        fos.rms_norm(x, w, rstd=torch.empty(9, device=DEV))
    with pytest.raises(fos.FosError):
        fos.rms_norm(x, w, eps=-1.0)
    with pytest.raises(fos.FosError):
        fos.rms_norm(x[:, :48].contiguous(), w[:48].contiguous())
    with pytest.raises(ValueError):
        fos.rms_norm(x, w, h=torch.empty_like(x))
    with pytest.raises(ValueError):
        fos.rms_norm_backward(x, x, rstd.half(), w)
    with pytest.raises(fos.FosError):
        fos.rms_norm_backward(x, x, rstd, w, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        fos.act_backward(x, x, "swish")
    with pytest.raises(ValueError):
        fos.act_backward(x, x.float(), "silu")
    with pytest.raises(fos.FosError):
        fos.act_backward(x, None, "silu")
    with pytest.raises(ValueError):
        fos.quantize8(x, scales=torch.empty(3, dtype=torch.uint8, device=DEV))
    with pytest.raises(fos.FosError) as e:
        fos._check(fos.lib().fos_quantize8(ctypes.c_void_p(x.data_ptr() + 2), 0, 8, 32, 1,
                                           ctypes.c_void_p(x.data_ptr()),
                                           ctypes.c_void_p(x.data_ptr()), None, None, None), "q")
    assert e.value.status == fos.FOS_ERR_MISALIGNED


def test_past_2_to_the_31_elements():
    """540,672 x 4096 (2.2e9 elements): the last rows of the norm and of both
    quantized forms equal those of the last rows alone."""
    R, C = 540672, 4096
    x = torch.empty(R, C, dtype=BF16, device=DEV)
    for r in range(0, R, 67584):
        x[r:r + 67584] = _rand(67584, C, BF16, r)
    w = torch.ones(C, device=DEV)
    tail = x[R - 256:].contiguous()
    got, one = fos.rms_norm(x, w, scale_tiled=False), fos.rms_norm(tail, w, scale_tiled=False)
    assert torch.equal(got[0][R - 256:], one[0]) and torch.equal(got[1][R - 256:], one[1])
    assert torch.equal(got[4][R - 256:], one[4])
    q, p = fos.quantize8(x, scale_tiled=False, colwise=True), fos.quantize8(tail, scale_tiled=False,
                                                                           colwise=True)
    assert torch.equal(q[0][R - 256:], p[0]) and torch.equal(q[2][:, R - 256:], p[2])
    assert torch.equal(q[1][R - 256:], p[1]) and torch.equal(q[3][:, (R - 256) // 32:], p[3])
