"""Rows packed by expert: the grouped products, the weight gradients, the grouped
8-bit quantization and the few-row product with NVFP4 weights, against plain 64-bit
forms (expert_reference).

Bounds, e = 2^-24, u = unit roundoff of the stored type, K terms of a sum:
  products  (K + 4) e sum |a b| (fp32 accumulation in any order, decode scales), then
            as in test_gpu_linear.py: bias one rounding, an activation's slope of at
            most 1.13 and 2^-20 of its argument, residual one rounding, u of the result
  matvec4   2 (K + 16) e sum |x w|: its accumulators may be truncated, which is two half
            steps; bf16 and fp32 rows are held to 2^-39 of the row's largest finite
            element, so 2^-39 max |x| sum |w| more
"""
import random

import pytest
import torch

import expert_reference as ex
import ffn_reference as ref
import nvfp4_quantization_precision_gb300 as fos

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = torch.float64
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV) * scale


def _offs(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _sizes(*n):
    out, e = [], 0
    for s in n:
        e += s
        out.append(e)
    return out


def _weights(fmt, w):
    """The experts' weights [G, N, K] as operands and their exact values."""
    codes, scales, amax, vals = [], [], [], []
    for e in range(w.shape[0]):
        N, K = w[e].shape
        if fmt == 8:
            c, s = fos.quantize8(w[e].contiguous())[:2]
            vals.append(ex.values8(c, ex.untile(s, N, K // 32)))
        else:
            c, s, a = fos.quantize(w[e].to(BF16).contiguous(), fos.Config(scale_tiled=True))
            amax.append(a)
            vals.append(ex.values4(c, ex.untile(s, N, K // 16)) * ex.decode_scale(a))
        codes.append(c)
        scales.append(s)
    return (torch.stack(codes), torch.stack(scales), torch.cat(amax) if amax else None), torch.stack(vals)


def _tokens(fmt, x, offs, row=False):
    """Packed rows as an operand and their exact values."""
    if fmt == 8:
        c, s = fos.quantize8(x, scale_tiled=False)[:2]
        return (c, s, None), ex.values8(c, s)
    if row:
        c, s, a = fos.quantize(x.to(BF16), fos.Config(row_scaled=True))
        return (c, s, a), ex.values4(c, s) * ex.decode_scale(a).unsqueeze(1)
    c, s, a = fos.quantize_grouped(x.to(BF16), _offs(offs))
    v = ex.values4(c, s)
    g = ex.decode_scale(a)
    for e, r0, r1, _, _ in ex.spans(offs, x.shape[0]):
        v[r0:r1] *= g[e]
    return (c, s, a), v


def _call(fmt, a, b, offs, row=False, **kw):
    if fmt == 8:
        return fos.linear8_grouped(a[0], a[1], b[0], b[1], _offs(offs), **kw)
    return fos.linear4_grouped(*a, *b, _offs(offs), cfg=fos.Config(row_scaled=row), **kw)


def _near(got, pre, av, wv, act, bias, residual, dt, factor=1.0, more=None):
    """One expert's rows against act(av . wv^T + bias) + residual."""
    K = av.shape[1]
    v = av @ wv.t()
    err = (av.abs() @ wv.abs().t()) * (factor * (K + 4) * 2.0 ** -24)
    if more is not None:
        err = err + more
    if bias is not None:
        v = v + bias.to(D)
        err = err + v.abs() * 2.0 ** -23
    if pre is not None:
        ref.near(pre, v, err + v.abs() * ref.U[dt] * (1 + 2.0 ** -10) + ref.TINY[dt], "pre")
    out = ref.act(v, act)
    if act != "none":
        err = 1.13 * err + v.abs() * 2.0 ** -20
    if residual is not None:
        out = out + residual.to(D)
        err = err + out.abs() * 2.0 ** -23
    ref.near(got, out, err * 1.01 + out.abs() * ref.U[dt] * (1 + 2.0 ** -10) + ref.TINY[dt], "out")


def _case(fmt, offs, rows, N, K, act="none", use_bias=False, res=False, pre=False, dt=BF16,
          row=False, bias32=True, seed=0):
    G = len(offs)
    b, wv = _weights(fmt, _rand(G, N, K, seed=seed + 1, scale=0.05))
    a, av = _tokens(fmt, _rand(rows, K, seed=seed + 2), offs, row)
    bias = _rand(G, N, seed=seed + 3) if use_bias else None
    if bias is not None and not bias32:
        bias = bias.to(dt)
    r = _rand(rows, N, seed=seed + 4).to(dt) if res else None
    out = torch.full((rows, N), 77.0, dtype=dt, device=DEV)
    kept = torch.full_like(out, 78.0) if pre else None
    got = _call(fmt, a, b, offs, row, act=act, bias=bias, residual=r, out_dtype=dt, save_pre=pre,
                out=out, pre=kept)
    out, p = got if pre else (got, None)
    for e, r0, r1, _, _ in ex.spans(offs, rows):
        if r1 > r0:
            _near(out[r0:r1], None if p is None else p[r0:r1], av[r0:r1], wv[e], act,
                  None if bias is None else bias[e], None if r is None else r[r0:r1], dt)
    end = ex.ends(offs, rows)[-1]
    assert (out[end:] == 77.0).all() and (p is None or (p[end:] == 78.0).all())
    return a, b


# experts that end inside every tile and box, with none, one and many rows
SIZES = [(1,), (3, 0, 1), (16, 15, 17), (31, 32, 33, 0), (96, 95, 97), (160, 161, 191, 192, 193),
         (0, 0, 5, 0), (384, 385, 2), (600,), (1, 1, 1, 1, 1, 1, 1, 1, 1)]


@pytest.mark.parametrize("fmt", [8, 4])
@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("N,K", [(16, 128), (272, 640), (1040, 1152)])
def test_grouped_sizes(fmt, sizes, N, K):
    offs = _sizes(*sizes)
    _case(fmt, offs, offs[-1] + 9, N, K, "silu", True, True, True, row=N == 272, seed=offs[-1])


@pytest.mark.parametrize("K", [64, 192, 256, 320, 448, 1088])
def test_grouped_nvfp4_ends_of_k(K):
    _case(4, _sizes(40, 0, 210), 260, 304, K, "none", True, False, False, F32)


@pytest.mark.parametrize("fmt", [8, 4])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_grouped_epilogues(fmt, act, dt):
    offs = _sizes(5, 130, 0, 70)
    for k, (b, r, p) in enumerate([(True, True, True), (False, False, False), (True, False, False),
                                   (False, True, False), (False, False, True)]):
        _case(fmt, offs, 205 + k, 336, 512, act, b, r, p, dt, row=k % 2 == 0, bias32=k == 0)


@pytest.mark.parametrize("fmt", [8, 4])
@pytest.mark.parametrize("sizes,N,K", [((3000, 100, 1), 512, 1024), ((20,) * 40, 768, 2048),
                                       ((700, 0, 900), 4096, 4096), ((64,) * 8, 256, 14336)])
def test_grouped_many_tiles(fmt, sizes, N, K):
    offs = _sizes(*sizes)
    _case(fmt, offs, offs[-1], N, K, "gelu_tanh", True, True, False)


@pytest.mark.parametrize("fmt", [8, 4])
@pytest.mark.parametrize("sizes", [(1,), (2, 0, 3, 1), (0, 0, 40, 0, 24), (17,), (1,) * 12])
@pytest.mark.parametrize("N,K", [(16, 8192), (144, 256), (336, 4224), (1104, 1664), (4096, 2048)])
def test_grouped_few_rows(fmt, sizes, N, K):
    """Few tiles: K in one part, two, four and eight."""
    offs = _sizes(*sizes)
    _case(fmt, offs, offs[-1] + 5, N, K, "gelu", True, True, True, (BF16, F16, F32)[(N // 16 + len(sizes)) % 3],
          row=N == 336, seed=N + len(sizes))


@pytest.mark.parametrize("fmt,sizes,N,K", [(8, (300, 5, 0, 550), 368, 15360), (4, (64, 65, 1, 128, 130), 96, 9280),
                                           (4, (256, 0, 255), 336, 8192), (8, (191, 63), 48, 4224)])
def test_grouped_few_tiles_of_many_rows(fmt, sizes, N, K):
    """Chunks of 64 rows, several of an expert and several of a cluster."""
    offs = _sizes(*sizes)
    _case(fmt, offs, offs[-1], N, K, "silu", True, True, False, row=True, seed=K)


@pytest.mark.parametrize("fmt", [8, 4])
@pytest.mark.parametrize("sizes,N,K", [((2, 0, 1), 320, 8192), ((1,) * 9, 1104, 5120), ((40, 24), 1024, 2048),
                                       ((400, 455), 368, 7680)])
def test_grouped_few_rows_many_calls_one_answer(fmt, sizes, N, K):
    offs, rows = _sizes(*sizes), sum(sizes)
    b, _ = _weights(fmt, _rand(len(sizes), N, K, seed=1))
    a, _ = _tokens(fmt, _rand(rows, K, seed=2), offs)
    res = _rand(rows, N, seed=3).to(BF16)
    want = _call(fmt, a, b, offs, act="silu", residual=res, out=res.clone())
    for _ in range(25):
        stream = res.clone()
        assert torch.equal(_call(fmt, a, b, offs, act="silu", residual=stream, out=stream), want)


@pytest.mark.parametrize("fmt", [8, 4])
@pytest.mark.parametrize("offs", [[5, 3, 9], [-4, 10, -7], [100, 200, 300], [0, 0, 0], [64, 64, 64],
                                  [2147483647, 0, 0]])
def test_ends_that_are_no_ends(fmt, offs):
    """Ends are clamped as the grouped quantizer clamps them."""
    _case(fmt, offs, 60, 144, 256, "relu", True, True, True)


@pytest.mark.parametrize("fmt", [8, 4])
def test_the_most_experts(fmt):
    r = random.Random(3)
    sizes = [r.choice((0, 0, 0, 0, 1, 2, 5)) for _ in range(1024)]
    offs = _sizes(*sizes)
    _case(fmt, offs, offs[-1] + 3, 32, 128, use_bias=True)
    with pytest.raises(fos.FosError) as e:
        _case(fmt, offs + [offs[-1]], offs[-1], 32, 128)
    assert e.value.status == fos.FOS_ERR_UNSUPPORTED


@pytest.mark.parametrize("fmt", [8, 4])
def test_other_experts_rows_do_not_matter(fmt):
    """NaN scales, and NaN or infinite epilogue operands, of rows beside an expert's and
    behind the last one change nothing in its rows."""
    offs, rows, N, K = _sizes(37, 0, 150), 230, 272, 512
    b, _ = _weights(fmt, _rand(3, N, K, seed=1))
    a, _ = _tokens(fmt, _rand(rows, K, seed=2), offs)
    res = _rand(rows, N, seed=3).to(BF16)
    want = _call(fmt, a, b, offs, residual=res, out=torch.zeros(rows, N, dtype=BF16, device=DEV))
    nan = 0xFF if fmt == 8 else 0x7F
    bad, res2 = a[1].clone(), res.clone()
    bad[0:37] = nan
    bad[187:] = nan
    res2[187:] = float("inf")
    got = _call(fmt, (a[0], bad, a[2]), b, offs, residual=res2,
                out=torch.zeros(rows, N, dtype=BF16, device=DEV))
    assert torch.isnan(got[:37]).all()
    assert torch.equal(got[37:], want[37:])
    # an expert's weights that are NaN reach its own rows alone
    ws = b[1].clone()
    ws[2] = nan
    got = _call(fmt, a, (b[0], ws, b[2]), offs, residual=res, out=torch.zeros_like(want))
    assert torch.equal(got[:37], want[:37]) and torch.isnan(got[37:187]).all()


def test_zero_amaxes_and_zero_rows():
    """An expert whose rows are all zeros gives its bias exactly."""
    offs, N, K = _sizes(20, 30), 64, 128
    x = _rand(50, K, seed=1)
    x[:20] = 0
    b, _ = _weights(4, _rand(2, N, K, seed=2))
    a, _ = _tokens(4, x, offs)
    bias = _rand(2, N, seed=3)
    got = _call(4, a, b, offs, bias=bias, out_dtype=F32)
    assert torch.equal(got[:20], bias[0].expand(20, N))


@pytest.mark.parametrize("fmt", [8, 4])
def test_grouped_in_place_and_repeats(fmt):
    offs, rows, N, K = _sizes(200, 33, 0, 411), 650, 1040, 2048
    b, _ = _weights(fmt, _rand(4, N, K, seed=1))
    a, _ = _tokens(fmt, _rand(rows, K, seed=2), offs)
    res = _rand(rows, N, seed=3).to(BF16)
    want = _call(fmt, a, b, offs, act="gelu", residual=res, out=res.clone())
    for _ in range(6):
        stream = res.clone()
        got = _call(fmt, a, b, offs, act="gelu", residual=stream, out=stream)
        assert got.data_ptr() == stream.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("fmt", [8, 4])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_grouped_residual_many_calls_one_answer(fmt, dt):
    """Many tiles with few stages: the residual's chunks run ahead over the ends of tiles, some
    of them without columns for a warp."""
    offs, rows, N, K = _sizes(*[(37 * e) % 211 for e in range(16)]), 1700, 2064, 384
    b, _ = _weights(fmt, _rand(16, N, K, seed=1))
    a, _ = _tokens(fmt, _rand(rows, K, seed=2), offs)
    res = _rand(rows, N, seed=3).to(dt)
    want = _call(fmt, a, b, offs, residual=res, out_dtype=dt, out=res.clone())
    for _ in range(25):
        stream = res.clone()
        assert torch.equal(_call(fmt, a, b, offs, residual=stream, out_dtype=dt, out=stream), want)


def test_side_stream_and_a_graph_for_every_routing():
    """One captured graph of quantization, product, gradient and weight gradient serves
    other ends than it was captured with."""
    rows, N, K, G = 300, 256, 384, 3
    w, _ = _weights(8, _rand(G, N, K, seed=1))
    x, pre = _rand(rows, K, seed=2).to(BF16), _rand(rows, N, seed=3).to(BF16)
    offs = _offs([100, 200, 300])

    def step(o):
        c, s, ct, st = fos.quantize8_grouped(x, o)
        y = fos.linear8_grouped(c, s, w[0], w[1], o, act="silu", out=torch.zeros(rows, N, dtype=BF16, device=DEV))
        dc, ds, dct, dst, d, db = fos.act_backward_grouped(y, pre, "silu", o)
        return y, fos.linear8_grouped_wgrad(dct, dst, ct, st, o, rows), db

    routings = [[100, 200, 300], [7, 7, 290], [0, 300, 300], [0, 0, 0]]
    want = [[t.clone() for t in step(_offs(r))] for r in routings]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(_offs(routings[1]))
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want[1]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(offs)
    for r, q in zip(routings, want):
        offs.copy_(_offs(r))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, q)), r


def test_grouped_outputs_past_2_to_the_31_elements():
    """150,000 x 14,336 outputs: an expert's rows at the end equal the product of them alone."""
    rows, N, K = 150000, 14336, 128
    offs = [70000, 149700, 150000]
    c, s = fos.quantize8(_rand(rows, K, seed=1), scale_tiled=False)[:2]
    b, _ = _weights(8, _rand(3, N, K, seed=2))
    out = fos.linear8_grouped(c, s, b[0], b[1], _offs(offs), act="relu")
    tail = fos.linear8_grouped(c[149700:], s[149700:], b[0][2:], b[1][2:], _offs([300]), act="relu")
    assert torch.equal(out[149700:], tail)


# ------------------------------------------------------------------ 8-bit quantization by expert
def _check_grouped8(q, x, offs, rows, cols):
    """Column-wise form against quantize8 of each expert's rows alone (tested itself)."""
    codes_t, scales_t = q
    P = ex.columns(rows, len(offs))
    assert fos.grouped_cols(rows, len(offs)) == P and codes_t.shape == (cols, P)
    sc = ex.untile(scales_t, cols, P // 32)
    for _, r0, r1, p0, p1 in ex.spans(offs, rows):
        if r1 == r0:
            continue
        _, _, ct, st = fos.quantize8(x[r0:r1].contiguous(), rowwise=False, colwise=True, scale_tiled=False)
        w = ct.shape[1]
        assert torch.equal(codes_t[:, p0:p0 + w], ct) and not codes_t[:, p0 + w:p1].any()
        assert torch.equal(sc[:, p0 // 32:(p0 + w) // 32], st) and not sc[:, (p0 + w) // 32:p1 // 32].any()


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("cols", [32, 160, 1024])
def test_quantize8_grouped(dt, sizes, cols):
    offs = _sizes(*sizes)
    rows = offs[-1] + 5
    x = _rand(rows, cols, seed=offs[-1]).to(dt)
    x[rows - 1, 0] = float("nan")
    P = ex.columns(rows, len(offs))
    n = (cols + 127) // 128 * (P // 128) * 512
    bufs = [torch.full(s, 0xAB, dtype=torch.uint8, device=DEV)
            for s in ((rows, cols), (rows, cols // 32), (cols, P), (n,))]
    c, s, ct, st = fos.quantize8_grouped(x, _offs(offs), codes=bufs[0], scales=bufs[1], codes_t=bufs[2],
                                         scales_t=bufs[3])
    end = offs[-1]
    wc, ws = fos.quantize8(x[:end].contiguous(), scale_tiled=False)[:2]
    assert torch.equal(c[:end], wc) and torch.equal(s[:end], ws)
    assert (c[end:] == 0xAB).all() and (s[end:] == 0xAB).all()
    _check_grouped8((ct, st), x, offs, rows, cols)
    p = ex.spans(offs, rows)[-1][4]
    assert (ct[:, p:] == 0xAB).all()
    # rows of padding of the tiled scales are zeros
    full = ex.untile(st, (cols + 127) // 128 * 128, P // 32)
    assert not full[cols:].any()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_act_backward_grouped(act, dt):
    """Codes, scales and d are those of act_backward (tested itself) of each expert's
    rows; dbias is the sum of the expert's d to n e sum |d|."""
    offs, rows, cols = _sizes(130, 0, 3, 257, 128), 530, 288
    dout, pre = _rand(rows, cols, seed=1).to(dt), _rand(rows, cols, seed=2, scale=2.0).to(dt)
    d0 = torch.full((rows, cols), 5.0, dtype=dt, device=DEV)
    db0 = torch.full((5, cols), float("nan"), device=DEV)
    c, s, ct, st, d, db = fos.act_backward_grouped(dout, None if act == "none" else pre, act, _offs(offs),
                                                   value=True, d=d0, dbias=db0)
    sc = ex.untile(st, cols, ct.shape[1] // 32)
    for e, r0, r1, p0, p1 in ex.spans(offs, rows):
        if r1 == r0:
            assert not db[e].any()
            continue
        wc, ws, wct, wst, wd, wdb = fos.act_backward(dout[r0:r1].contiguous(),
                                                     None if act == "none" else pre[r0:r1].contiguous(), act,
                                                     scale_tiled=False, value=True)
        assert torch.equal(c[r0:r1], wc) and torch.equal(s[r0:r1], ws) and torch.equal(d[r0:r1], wd)
        w = wct.shape[1]
        assert torch.equal(ct[:, p0:p0 + w], wct) and torch.equal(sc[:, p0 // 32:(p0 + w) // 32], wst)
        assert not ct[:, p0 + w:p1].any()
        v = dout[r0:r1].to(D) * (ref.act_slope(pre[r0:r1].to(D), act) if act != "none" else 1.0)
        # the derivative's own error (test_gpu_ffn_numerics.py) and the sum's
        near = (r1 - r0) * 2.0 ** -24 * v.abs().sum(0) + (dout[r0:r1].to(D).abs() * 2.0 ** -20).sum(0)
        ref.near(db[e], v.sum(0), near + 1e-30, "dbias")
        ref.near(db[e], wdb.to(D), 2 * (r1 - r0) * 2.0 ** -24 * v.abs().sum(0) + 1e-30, "dbias alone")
    assert (d[518:] == 5.0).all()


def test_act_backward_grouped_parts_and_places():
    """Each output alone equals itself among all; d in the place of dout or of pre."""
    offs, rows, cols = _sizes(100, 200), 300, 256
    dout, pre = _rand(rows, cols, seed=1).to(BF16), _rand(rows, cols, seed=2).to(BF16)
    o = _offs(offs)
    c, s, ct, st, d, db = fos.act_backward_grouped(dout, pre, "gelu", o, value=True)
    for kw in (dict(rowwise=True, colwise=False, bias_grad=False), dict(rowwise=False, bias_grad=False),
               dict(rowwise=False, colwise=False), dict(rowwise=False, colwise=False, bias_grad=False, value=True)):
        got = fos.act_backward_grouped(dout, pre, "gelu", o, **kw)
        for p, q in zip(got, (c, s, ct, st, d, db)):
            # the last expert's part ends the column-wise form here
            assert p is None or torch.equal(p[:, :384] if p is got[2] else p, q[:, :384] if p is got[2] else q) \
                or p is got[3]
        if got[2] is not None:
            assert torch.equal(ex.untile(got[3], cols, ct.shape[1] // 32)[:, :12],
                               ex.untile(st, cols, ct.shape[1] // 32)[:, :12])
    for which in (0, 1):
        t = [dout.clone(), pre.clone()]
        got = fos.act_backward_grouped(t[0], t[1], "gelu", o, value=True, d=t[which])
        assert torch.equal(got[4], d) and torch.equal(got[0], c) and torch.equal(got[5], db)


def test_grouped_quantization_of_nothing():
    x = torch.empty(0, 64, dtype=BF16, device=DEV)
    c, s, ct, st = fos.quantize8_grouped(x, _offs([0, 0]))
    assert c.shape == (0, 64) and ct.shape == (64, 0)
    db = fos.act_backward_grouped(x, x, "relu", _offs([0, 0]))[5]
    assert db.shape == (2, 64) and not db.any()
    e = torch.empty(0, 128, dtype=torch.uint8, device=DEV)
    w, _ = _weights(8, _rand(2, 16, 128, seed=1))
    y = fos.linear8_grouped(e, torch.empty(0, 4, dtype=torch.uint8, device=DEV), w[0], w[1], _offs([0, 0]))
    assert y.shape == (0, 16)


def test_columns_past_2_to_the_31():
    """16,384 x 140,032 column-wise codes (2.29e9): the last expert's equal its own alone."""
    rows, cols = 140000, 16384
    offs = [60000, 139800, 140000]
    x = _rand(rows, cols, seed=1, scale=0.5).to(BF16)
    ct, st = fos.quantize8_grouped(x, _offs(offs), rowwise=False)[2:]
    p0 = ex.spans(offs, rows)[2][3]
    want = fos.quantize8(x[139800:].contiguous(), rowwise=False, colwise=True, scale_tiled=False)[2]
    assert torch.equal(ct[:, p0:p0 + want.shape[1]], want)


# ------------------------------------------------------------------ weight gradients
def _wgrad(offs, rows, N, K, dt, res, seed=0, inplace=False, cut=False):
    d, z = _rand(rows, N, seed=seed + 1).to(BF16), _rand(rows, K, seed=seed + 2).to(BF16)
    o = _offs(offs)
    dct, dst = fos.quantize8_grouped(d, o, rowwise=False)[2:]
    zct, zst = fos.quantize8_grouped(z, o, rowwise=False)[2:]
    if cut:  # without the last 16 columns of both (the scales' rows come to whole tiles all the same)
        N, K = N - 16, K - 16
        dct, zct = dct[:N], zct[:K]
    G, P = len(offs), dct.shape[1]
    r = _rand(G, N, K, seed=seed + 3).to(dt) if res else None
    out = r.clone() if inplace else torch.full((G, N, K), float("nan"), dtype=dt, device=DEV)
    got = fos.linear8_grouped_wgrad(dct, dst, zct, zst, o, rows, residual=out if inplace else r,
                                    out_dtype=dt, out=out)
    dv = ex.values8(dct, ex.untile(dst, N, P // 32))
    zv = ex.values8(zct, ex.untile(zst, K, P // 32))
    for e, r0, r1, p0, p1 in ex.spans(offs, rows):
        a, b = dv[:, p0:p1], zv[:, p0:p1]
        want = a @ b.t()
        err = (a.abs() @ b.abs().t()) * ((p1 - p0 + 4) * 2.0 ** -24)
        if res:
            want = want + r[e].to(D)
            err = err + want.abs() * 2.0 ** -23
        ref.near(got[e], want, err * 1.01 + want.abs() * ref.U[dt] * (1 + 2.0 ** -10) + ref.TINY[dt], "dW")
        if r1 == r0 and not res:
            assert not got[e].any()


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("N,K", [(32, 32), (288, 672), (1056, 256)])
def test_wgrad_sizes(sizes, N, K):
    offs = _sizes(*sizes)
    _wgrad(offs, offs[-1] + 7, N, K, F32, False, seed=offs[-1])


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("res", [False, True])
def test_wgrad_types(dt, res):
    _wgrad(_sizes(300, 0, 129, 700), 1200, 544, 800, dt, res)
    if res:
        _wgrad(_sizes(0, 150, 129), 279, 544, 800, dt, True, inplace=True)


@pytest.mark.parametrize("offs,rows", [([5, 3, 9], 60), ([0, 0, 0], 40), ([-1, 90, 400], 120), ([2500, 2600, 6000], 6000)])
def test_wgrad_ends(offs, rows):
    _wgrad(offs, rows, 320, 416, F32, True)


def test_wgrad_of_no_rows():
    w = torch.full((2, 32, 64), 3.0, device=DEV)
    e = torch.empty(32, 0, dtype=torch.uint8, device=DEV), torch.empty(64, 0, dtype=torch.uint8, device=DEV)
    n = torch.empty(0, dtype=torch.uint8, device=DEV)
    got = fos.linear8_grouped_wgrad(e[0], n, e[1], n, _offs([0, 0]), 0, residual=w)
    assert torch.equal(got, w) and got.data_ptr() != w.data_ptr()
    assert not fos.linear8_grouped_wgrad(e[0], n, e[1], n, _offs([0, 0]), 0).any()


def test_wgrad_many_calls_one_answer():
    """Many tiles with few stages each, back to back: every repeat equals the first."""
    offs, rows, N, K = _sizes(863, 835, 0, 822, 789), 3400, 4096, 2048
    o = _offs(offs)
    dct, dst = fos.quantize8_grouped(_rand(rows, N, seed=1, scale=0.05).to(BF16), o, rowwise=False)[2:]
    zct, zst = fos.quantize8_grouped(_rand(rows, K, seed=2).to(BF16), o, rowwise=False)[2:]
    one = fos.linear8_grouped_wgrad(dct, dst, zct, zst, o, rows)
    for _ in range(12):
        assert torch.equal(one, fos.linear8_grouped_wgrad(dct, dst, zct, zst, o, rows))


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("N,K", [(64, 224), (288, 416), (416, 1024)])
def test_wgrad_residual_over_tile_ends(dt, N, K):
    """More tiles than pairs of SMs, with rows that fill no, one or some of a tile's row
    chunks: the residual's chunks are fetched ahead of the tile that adds them."""
    sizes = [(7 * e * e + 3 * e) % 67 for e in range(200)]
    offs = _sizes(*sizes)
    _wgrad(offs, offs[-1], N, K, dt, True, seed=N, inplace=True, cut=True)


@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_wgrad_rows_that_end_inside_a_chunk(dt):
    """16 more rows than whole chunks of 32: the next expert's rows stay its own."""
    _wgrad(_sizes(300, 0, 129, 40), 480, 288, 416, dt, False, cut=True)


def test_wgrad_with_residual_many_calls_one_answer():
    offs, rows, N, K = _sizes(*[(5 * e) % 23 for e in range(64)]), 700, 1056, 672
    o = _offs(offs)
    dct, dst = fos.quantize8_grouped(_rand(rows, N, seed=1).to(BF16), o, rowwise=False)[2:]
    zct, zst = fos.quantize8_grouped(_rand(rows, K, seed=2).to(BF16), o, rowwise=False)[2:]
    r = _rand(64, N, K, seed=3)
    one = fos.linear8_grouped_wgrad(dct, dst, zct, zst, o, rows, residual=r)
    for _ in range(20):
        assert torch.equal(one, fos.linear8_grouped_wgrad(dct, dst, zct, zst, o, rows, residual=r))


def test_gradients_against_differences():
    """The product is linear in both operands: with small whole numbers every product
    is exact, and so are the differences of sum(g * out) by one element."""
    offs, rows, N, K, G = _sizes(33, 0, 50), 83, 64, 128, 3
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    whole = lambda *s: torch.randint(-4, 5, s, generator=gen, device=DEV).float()  # noqa: E731
    x, w, g = whole(rows, K), whole(G, N, K), whole(rows, N)
    o = _offs(offs)

    def loss(xx, ww):
        c, s = fos.quantize8(xx, scale_tiled=False)[:2]
        b = _weights(8, ww)[0]
        return (fos.linear8_grouped(c, s, b[0], b[1], o, out_dtype=F32) * g).sum(dtype=D)

    gct, gst = fos.quantize8_grouped(g, o, rowwise=False)[2:]
    xct, xst = fos.quantize8_grouped(x, o, rowwise=False)[2:]
    dw = fos.linear8_grouped_wgrad(gct, gst, xct, xst, o, rows)
    wt = [fos.quantize8(w[e].contiguous(), rowwise=False, colwise=True)[2:] for e in range(G)]
    # the input gradient's K is N here, a multiple of 128 by zero columns
    gp = torch.zeros(rows, 128, device=DEV)
    gp[:, :N] = g
    wtc = torch.zeros(G, K, 128, dtype=torch.uint8, device=DEV)
    wts = torch.zeros(G, 512, dtype=torch.uint8, device=DEV)
    for e in range(G):
        wtc[e, :, :N] = wt[e][0]
        wts[e] = wt[e][1]
    gc, gs = fos.quantize8(gp, scale_tiled=False)[:2]
    dx = fos.linear8_grouped(gc, gs, wtc, wts, o, out_dtype=F32)
    base = loss(x, w)
    for e, n, k in ((0, 3, 7), (0, 63, 127), (1, 5, 5), (2, 0, 0), (2, 40, 99)):
        ww = w.clone()
        ww[e, n, k] += 1
        assert float(loss(x, ww) - base) == float(dw[e, n, k])
    for r, k in ((0, 0), (32, 5), (33, 127), (82, 64)):
        xx = x.clone()
        xx[r, k] += 1
        assert float(loss(xx, w) - base) == float(dx[r, k])


# ------------------------------------------------------------------ few rows, NVFP4 weights
def _matvec(M, X, G, N, K, dt=BF16, out_dt=None, act="none", use_bias=False, res=False, ids=None,
            x=None, seed=0, bias32=True, bound=448):
    out_dt = dt if out_dt is None else out_dt
    cfg = fos.Config(scale_tiled=True, bound=bound)
    n = max(G, 1)
    codes, scales, amax, wv = [], [], [], []
    for e in range(n):
        c, s, a = fos.quantize(_rand(N, K, seed=seed + 10 + e, scale=0.05).to(BF16), cfg)
        S = torch.tensor(6.0 * bound) / a.cpu()
        wv.append(ex.values4(c, ex.untile(s, N, K // 16)) * (1 / S).to(D).to(DEV))
        codes.append(c)
        scales.append(s)
        amax.append(a)
    x = _rand(X, K, seed=seed + 1).to(dt) if x is None else x
    b = (torch.stack(codes), torch.stack(scales), torch.cat(amax)) if G else (codes[0], scales[0], amax[0])
    bias = _rand(n, N, seed=seed + 2) if use_bias else None
    if bias is not None:
        bias = bias if bias32 else bias.to(out_dt)
        bias = bias if G else bias[0]
    r = _rand(M, N, seed=seed + 3).to(out_dt) if res else None
    out = torch.full((M, N), 77.0, dtype=out_dt, device=DEV)
    got = fos.matvec4(x, *b, ids=None if ids is None else _offs(ids), act=act, bias=bias, residual=r,
                      out_dtype=out_dt, cfg=cfg, out=out)
    for p in range(M):
        e = 0 if ids is None else ids[p]
        if not 0 <= e < n:
            assert (got[p] == 77.0).all()
            continue
        xv = x[p // (M // X):p // (M // X) + 1].to(D)
        more = 2.0 ** -39 * xv.abs().max() * wv[e].abs().sum(1) if dt != F16 else None
        _near(got[p:p + 1], None, xv, wv[e], act, None if bias is None else (bias[e] if G else bias),
              None if r is None else r[p:p + 1], out_dt, 2.0 * (K + 16) / (K + 4), more)
    return got


# rows around the chunks of eight (two for fp32), weights and K inside every tile and split
@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("M", [1, 2, 3, 7, 8, 9, 17])
@pytest.mark.parametrize("N,K", [(16, 32), (144, 160), (1040, 1056)])
def test_matvec_sizes(dt, M, N, K):
    _matvec(M, M, 0, N, K, dt, act="silu", use_bias=True, res=True, seed=M + N)


@pytest.mark.parametrize("M,N,K", [(1, 14336, 4096), (1, 4096, 14336), (8, 256, 16384), (5, 2048, 7168),
                                   (1, 16384, 288), (3, 7168, 2048), (40, 512, 1024)])
def test_matvec_shapes_and_splits(M, N, K):
    _matvec(M, M, 0, N, K, act="gelu", use_bias=True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt,out_dt", [(BF16, F32), (F16, BF16), (F32, F16), (F32, F32)])
def test_matvec_epilogues(act, dt, out_dt):
    for b, r in ((True, True), (False, False), (True, False), (False, True)):
        _matvec(4, 4, 0, 208, 320, dt, out_dt, act, b, r, bias32=r, bound=256 if r else 448)


@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_matvec_experts(dt):
    _matvec(6, 3, 4, 272, 256, dt, act="relu", use_bias=True, res=True, ids=[2, 0, 2, 3, 0, 2])
    # ids that are no experts, one expert alone, more of its rows than a chunk
    _matvec(5, 5, 3, 64, 128, dt, use_bias=True, ids=[-1, 2, 3, 2, 7])
    _matvec(40, 20, 2, 144, 512, dt, use_bias=True, ids=[(p * 7) % 5 % 2 for p in range(40)])
    _matvec(4, 1, 16, 528, 1056, dt, ids=[15, 3, 8, 0])
    _matvec(3, 3, 2, 32, 64, dt, ids=[5, -3, 9])


def test_matvec_most_rows():
    r = random.Random(1)
    _matvec(1024, 256, 64, 16, 32, ids=[r.randrange(-1, 64) for _ in range(1024)])
    _matvec(1024, 1024, 0, 32, 64)
    x = torch.zeros(1025, 64, dtype=BF16, device=DEV)
    c, s, a = fos.quantize(_rand(32, 64, seed=1).to(BF16), fos.Config(scale_tiled=True))
    with pytest.raises(fos.FosError) as e:
        fos.matvec4(x, c, s, a)
    assert e.value.status == fos.FOS_ERR_UNSUPPORTED


@pytest.mark.parametrize("dt", [BF16, F32])
def test_matvec_range_of_x(dt):
    """Rows of very large, very small and mixed magnitudes, subnormal ones, zeros."""
    K = 512
    base = _rand(6, K, seed=3)
    base[0] *= 1e36
    base[1] *= 1e-36
    base[2] *= torch.pow(10.0, torch.linspace(-30, 30, K, device=DEV))
    base[3] *= 2.0 ** -128
    base[4] = 0
    base[5, 1:] = 0
    _matvec(6, 6, 0, 80, K, dt, F32, x=base.to(dt))
    top = torch.finfo(dt).max
    x = torch.zeros(1, K, dtype=dt, device=DEV)
    x[0, 5], x[0, 300] = top, -top
    _matvec(1, 1, 0, 16, K, dt, F32, x=x * 0.001 if dt == F32 else (x.float() * 0.001).to(dt))


def test_matvec_fp32_is_fp32():
    """24-bit elements: nothing of them is dropped (whole numbers below 2^24 with
    powers of two as weights are exact)."""
    K = 256
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randint(-(1 << 23), 1 << 23, (2, K), generator=g, device=DEV).float() * 2 + 1
    w = torch.zeros(16, K, device=DEV)
    for n in range(16):
        w[n, 16 * n % K] = 6.0  # amax 6: decode scale 6 / 2688 exactly undone
        w[n, (16 * n + 3) % K] = 3.0
    c, s, a = fos.quantize(w, fos.Config(scale_tiled=True))
    got = fos.matvec4(x, c, s, a)
    want = (x.to(D) @ w.to(D).t())
    # two terms: a product each with the decode scale, one sum
    assert ((got.to(D) - want).abs() <= want.abs() * 2.0 ** -22 + (x.abs().max() * 9) * 2.0 ** -24).all()


@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_matvec_infinities_and_nan(dt):
    """An infinity or a NaN in a row of x reaches its own outputs as in the formula: an
    infinity of the sign that the weight gives it, finite elements beside it intact."""
    K, N = 256, 48
    c, s, a = fos.quantize(_rand(N, K, seed=1).to(BF16), fos.Config(scale_tiled=True))
    wv = ex.values4(c, ex.untile(s, N, K // 16))
    x = _rand(4, K, seed=2).to(dt)
    clean = fos.matvec4(x, c, s, a)
    x[1, 7], x[2, 9] = float("inf"), float("nan")
    got = fos.matvec4(x, c, s, a).float()
    assert torch.equal(got[0], clean[0].float()) and torch.equal(got[3], clean[3].float())
    assert torch.isnan(got[2]).all()
    w7 = wv[:, 7]
    assert torch.isnan(got[1][w7 == 0]).all()
    assert (got[1][w7 > 0] == float("inf")).all() and (got[1][w7 < 0] == float("-inf")).all()


def test_matvec_nan_scale_and_zero_amax():
    K, N = 128, 32
    c, s, a = fos.quantize(_rand(N, K, seed=1).to(BF16), fos.Config(scale_tiled=True))
    x = _rand(2, K, seed=2).to(BF16)
    bad = s.clone()
    bad[int(ref.tile_index(N, K // 16)[5, 3])] = 0x7F
    got, want = fos.matvec4(x, c, bad, a), fos.matvec4(x, c, s, a)
    assert torch.isnan(got[:, 5]).all()
    got[:, 5] = want[:, 5]
    assert torch.equal(got, want)
    zc, zs, za = fos.quantize(torch.zeros(N, K, dtype=BF16, device=DEV), fos.Config(scale_tiled=True))
    assert not fos.matvec4(x, zc, zs, za).any()


def test_matvec_repeats_streams_graphs():
    ids = [3, 1, 3, 0, 2, 1, 1, 3]
    w = [fos.quantize(_rand(1040, 2048, seed=e).to(BF16), fos.Config(scale_tiled=True)) for e in range(4)]
    b = [torch.stack([t[0] for t in w]), torch.stack([t[1] for t in w]), torch.cat([t[2] for t in w])]
    x, i = _rand(8, 2048, seed=9).to(BF16), _offs(ids)
    want = fos.matvec4(x, *b, ids=i)
    for _ in range(10):
        assert torch.equal(want, fos.matvec4(x, *b, ids=i))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = fos.matvec4(x, *b, ids=i)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fos.matvec4(x, *b, ids=i, out=out)
    for r in (ids, ids[::-1], [0] * 8):
        i.copy_(_offs(r))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, fos.matvec4(x, *b, ids=_offs(r)))


@pytest.mark.parametrize("M,N,K", [(1, 14336, 4096), (2, 4096, 14336), (8, 2048, 7168)])
def test_matvec_many_calls_one_answer(M, N, K):
    """The rings of codes are filled again while their warps work: every repeat equals the first."""
    c, s, a = fos.quantize(_rand(N, K, seed=1).to(BF16), fos.Config(scale_tiled=True))
    x = _rand(M, K, seed=2).to(BF16)
    one = fos.matvec4(x, c, s, a, out_dtype=F32)
    outs = [fos.matvec4(x, c, s, a, out_dtype=F32) for _ in range(60)]
    assert all(torch.equal(one, o) for o in outs)


# ------------------------------------------------------------------ refusals
def test_refusals():
    w, _ = _weights(8, _rand(2, 64, 128, seed=1))
    c, s = fos.quantize8(_rand(10, 128, seed=2), scale_tiled=False)[:2]
    o = _offs([4, 10])
    fos.linear8_grouped(c, s, w[0], w[1], o)
    for args, kw in [((c, s, w[0], w[1], o.long()), {}), ((c, s, w[0], w[1], o.cpu()), {}),
                     ((c, s, w[0], w[1], _offs([10])), {}), ((c, s[:9], w[0], w[1], o), {}),
                     ((c, s, w[0], w[1][:, :-1], o), {}), ((c, s, w[0][0], w[1], o), {}),
                     ((c[:, :64], s, w[0], w[1], o), {}),
                     ((c, s, w[0], w[1], o), dict(bias=torch.ones(64, device=DEV))),
                     ((c, s, w[0], w[1], o), dict(residual=torch.ones(10, 64, device=DEV))),
                     ((c, s, w[0], w[1], o), dict(act="tanh"))]:
        with pytest.raises(ValueError):
            fos.linear8_grouped(*args, **kw)
    w96, _ = _weights(8, _rand(2, 64, 96, seed=1))
    c96, s96 = fos.quantize8(_rand(10, 96, seed=2), scale_tiled=False)[:2]
    with pytest.raises(fos.FosError) as e:
        fos.linear8_grouped(c96, s96, w96[0], w96[1], o)
    assert e.value.status == fos.FOS_ERR_UNSUPPORTED
    res = torch.zeros(11, 64, dtype=BF16, device=DEV)
    with pytest.raises(fos.FosError) as e:  # out over part of the residual
        fos.linear8_grouped(c, s, w[0], w[1], o, residual=res[:10], out=res[1:])
    assert e.value.status == fos.FOS_ERR_INVALID_ARG
    x = _rand(10, 64, seed=3).to(BF16)
    for call in (lambda: fos.quantize8_grouped(x, o.float()), lambda: fos.quantize8_grouped(x[0], o),
                 lambda: fos.act_backward_grouped(x, x[:5], "relu", o),
                 lambda: fos.linear8_grouped_wgrad(c.t().contiguous(), s, c, s, o, 10),
                 lambda: fos.matvec4(x, c, s, torch.ones(1, device=DEV)),
                 lambda: fos.grouped_cols(-1, 4), lambda: fos.grouped_cols(4, 0)):
        with pytest.raises(ValueError):
            call()
    m, sm, am = fos.quantize(_rand(32, 64, seed=1).to(BF16), fos.Config(scale_tiled=True))
    with pytest.raises(fos.FosError) as e:  # ids no multiple of the rows of x
        fos.matvec4(x[:2], m.unsqueeze(0), sm.unsqueeze(0), am, ids=_offs([0, 0, 0]))
    assert e.value.status == fos.FOS_ERR_INVALID_ARG


def test_moe_block_example():
    """The example's training step, served batch and served tokens: results of quantized
    operands lie within a few hundredths (8 bit), two or three tenths (NVFP4 on both sides),
    a tenth and a half (NVFP4 weights) of the unquantized block's."""
    import importlib.util
    import os
    p = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", p)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    for tokens, experts, act in ((77, 4, "silu"), (5, 16, "gelu")):
        err = m.run(tokens, 256, 384, experts, act=act)
        for k, v in err.items():
            assert v < (0.3 if "batch" in k else 0.2 if "tokens" in k else 0.1), (k, v)
