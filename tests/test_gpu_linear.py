"""The products with an epilogue (linear8, linear4) against plain 64-bit forms
(ffn_reference), over formats, output types, activations, token counts from
one, ragged sizes, long K, special values; repeats bit for bit; refusals.

Bound of one output, e = 2^-24, u = unit roundoff of the stored type, K terms:
  product  gamma_(K+2) sum |a b| (fp32 accumulation in any order)
  bias     one rounding, e |v|
  act      the slope is at most 1.13, so 1.13 times the above, plus the
           activation's own error: at most 2^-20 |v| (exp, erf within 2 ulp,
           four roundings; gelu and silu are v times a factor in [0, 1])
  residual one rounding, then u |out|
"""
import pytest
import torch

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


def _rand(rows, cols, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(rows, cols, generator=g, device=DEV) * scale


def _operand(fmt, x, row=False):
    """(codes, tiled scales, amax or None) and the exact values in doubles."""
    R, K = x.shape
    if fmt == 8:
        c, s, _, _ = fos.quantize8(x)
        sc = ref.untile(s, R, K // 32).long()
        v = (ref.blocks(ref.e4m3(c)) * ref.pow2(sc - 127).unsqueeze(2)).reshape(R, K)
        return (c, s, None), v.to(DEV)
    cfg = fos.Config(row_scaled=row, scale_tiled=True)
    c, s, a = fos.quantize(x.to(BF16), cfg)
    t = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=D)
    cc = c.cpu().long()
    v = torch.stack((t[cc & 15], t[cc >> 4]), 2).reshape(R, K // 16, 16)
    v = (v * ref.e4m3(ref.untile(s, R, K // 16)).unsqueeze(2)).reshape(R, K)
    S = torch.tensor(2688.0) / a.cpu()
    g = torch.where(a.cpu() > 0, 1 / S, torch.ones_like(S)).to(D)
    return (c, s, a), (v * g.unsqueeze(1)).to(DEV)


def _call(fmt, a, b, row=False, **kw):
    if fmt == 8:
        return fos.linear8(a[0], a[1], b[0], b[1], **kw)
    return fos.linear4(a[0], a[1], a[2], b[0], b[1], b[2], cfg=fos.Config(row_scaled=row), **kw)


def _check(got, pre, av, bv, act, bias, residual, dt):
    K = av.shape[1]
    v = av @ bv.t()
    err = (av.abs() @ bv.abs().t()) * ((K + 4) * 2.0 ** -24)
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


def _case(fmt, M, N, K, act="none", use_bias=False, res=False, pre=False, dt=BF16, row=False,
          bias32=True, seed=0):
    a, av = _operand(fmt, _rand(M, K, seed + 1), row)
    b, bv = _operand(fmt, _rand(N, K, seed + 2, 0.05))
    bias = _rand(1, N, 3)[0] if use_bias else None
    if bias is not None and not bias32:
        bias = bias.to(dt)
    r = _rand(M, N, 4).to(dt) if res else None
    out = torch.full((M, N), float("nan"), dtype=dt, device=DEV)
    got = _call(fmt, a, b, row, act=act, bias=bias, residual=r, out_dtype=dt, save_pre=pre, out=out)
    out, p = got if pre else (got, None)
    _check(out, p, av, bv, act, bias, r, dt)
    return a, b


# token counts around every tile size, weights and K that end inside a tile
@pytest.mark.parametrize("fmt", [8, 4])
@pytest.mark.parametrize("M,N,K", [
    (1, 16, 32), (1, 128, 128), (1, 4096, 4096), (2, 144, 160), (15, 256, 256), (16, 272, 288),
    (17, 1040, 1056), (48, 4096, 1024), (64, 128, 8192), (100, 2048, 512), (127, 400, 96),
    (128, 384, 64), (129, 192, 2080), (200, 512, 4128), (255, 1024, 1024), (256, 256, 256),
    (257, 256, 512), (300, 304, 320), (511, 1152, 1024), (513, 768, 96), (1000, 2064, 1056)])
def test_sizes(fmt, M, N, K):
    _case(fmt, M, N, K, "silu", True, True, True, row=M % 2 == 1, seed=M + N + K)


@pytest.mark.parametrize("fmt", [8, 4])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_epilogues(fmt, act, dt):
    for M in (3, 140, 600):
        _case(fmt, M, 336, 512, act, True, True, True, dt, row=True, bias32=M == 3)
        _case(fmt, M, 336, 512, act, False, False, False, dt)
        _case(fmt, M, 336, 512, act, True, False, False, dt)
        _case(fmt, M, 336, 512, act, False, True, False, dt, row=True)
        _case(fmt, M, 336, 512, act, False, False, True, dt)


@pytest.mark.parametrize("fmt", [8, 4])
@pytest.mark.parametrize("M,N,K", [(1, 256, 16384), (7, 14336, 512), (40, 4096, 14336),
                                   (300, 1024, 16384), (700, 4096, 4096), (2049, 2048, 1024)])
def test_long_and_wide(fmt, M, N, K):
    _case(fmt, M, N, K, "gelu_tanh", True, True, False, row=True)


@pytest.mark.parametrize("fmt", [8, 4])
def test_plain_product_equals_mm_or_the_exact_one(fmt):
    """No epilogue, fp32 out: NVFP4 equals fos.mm's bound; small integers are exact."""
    M, N, K = 80, 160, 256
    if fmt == 8:
        g = torch.Generator(device=DEV)
        g.manual_seed(1)
        x = torch.randint(-8, 9, (M, K), generator=g, device=DEV).float()
        w = torch.randint(-8, 9, (N, K), generator=g, device=DEV).float()
        a, _ = _operand(8, x)
        b, _ = _operand(8, w)
        got = _call(8, a, b, out_dtype=F32)
        assert torch.equal(got.to(D), x.to(D) @ w.to(D).t())
    else:
        a, av = _operand(4, _rand(M, K, 1))
        b, bv = _operand(4, _rand(N, K, 2))
        got = _call(4, a, b, out_dtype=F32)
        mm = fos.mm(a[0], a[1], a[2], b[0], b[1], b[2])
        lim = (av.abs() @ bv.abs().t()) * (2 * (K + 4) * 2.0 ** -24)
        ref.near(got, mm.to(D), lim, "fos.mm")


@pytest.mark.parametrize("fmt", [8, 4])
def test_nan_and_infinite_entries_stay_in_their_rows(fmt):
    """A NaN scale in one token's row, an infinity and a NaN in the residual."""
    for M in (5, 300):
        a, av = _operand(fmt, _rand(M, 256, 1))
        b, bv = _operand(fmt, _rand(160, 256, 2))
        bad = a[1].clone()
        # scale of row 2, block 1: 0xFF is NaN as UE8M0, 0x7F as E4M3
        bad[int(ref.tile_index(M, 256 // (32 if fmt == 8 else 16))[2, 1])] = 0xFF if fmt == 8 else 0x7F
        res = _rand(M, 160, 3).to(BF16)
        res[4, 7], res[3, 9] = float("inf"), float("nan")
        got = _call(fmt, (a[0], bad, a[2]), b, residual=res)
        assert torch.isnan(got[2]).all()
        assert torch.isinf(got[4, 7]) and torch.isnan(got[3, 9])
        got[2], got[4, 7], got[3, 9] = 0, 0, 0
        assert torch.isfinite(got).all()


@pytest.mark.parametrize("fmt", [8, 4])
def test_zero_rows_give_bias_and_residual(fmt):
    x = _rand(20, 128, 1)
    x[3:9] = 0
    a, av = _operand(fmt, x, True)
    b, bv = _operand(fmt, _rand(64, 128, 2))
    bias, res = _rand(1, 64, 3)[0], _rand(20, 64, 4)
    got = _call(fmt, a, b, True, bias=bias, residual=res, out_dtype=F32)
    assert torch.equal(got[3:9], (bias + res)[3:9])


@pytest.mark.parametrize("fmt", [8, 4])
@pytest.mark.parametrize("M", [1, 50, 1500])
def test_two_calls_one_answer(fmt, M):
    a, _ = _operand(fmt, _rand(M, 4096, 1))
    b, _ = _operand(fmt, _rand(2048, 4096, 2))
    one = _call(fmt, a, b, act="gelu")
    for _ in range(3):
        assert torch.equal(one, _call(fmt, a, b, act="gelu"))


@pytest.mark.parametrize("fmt", [8, 4])
def test_side_stream_and_graph(fmt):
    a, _ = _operand(fmt, _rand(33, 1024, 1))
    b, _ = _operand(fmt, _rand(512, 1024, 2))
    want = _call(fmt, a, b, act="relu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = _call(fmt, a, b, act="relu")
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _call(fmt, a, b, act="relu", out=out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_operands_of_the_norm_and_of_the_columns():
    """The norm's codes are an operand as they are; codes_t give the transposed
    products, over a ragged number of tokens."""
    T, C, N = 300, 512, 384
    x, w = _rand(T, C, 1).to(BF16), torch.ones(C, device=DEV)
    codes, scales, _, _, _ = fos.rms_norm(x, w)
    bw = _rand(N, C, 2, 0.05).to(BF16)
    bc, bs, bct, bst = fos.quantize8(bw, colwise=True)
    out = fos.linear8(codes, scales, bc, bs, out_dtype=F32)

    def dec(c, s):
        R, K = c.shape
        sc = ref.untile(s, R, K // 32).long()
        return (ref.blocks(ref.e4m3(c)) * ref.pow2(sc - 127).unsqueeze(2)).reshape(R, K).to(DEV)

    _check(out, None, dec(codes, scales), dec(bc, bs), "none", None, None, F32)
    dout = _rand(T, N, 3, 0.1).to(BF16)
    dc, ds, dct, dst, _, _ = fos.act_backward(dout, None, "none")
    xc, xs, xct, xst = fos.quantize8(x, colwise=True)
    da = fos.linear8(dc, ds, bct, bst, out_dtype=F32)
    _check(da, None, dec(dc, ds), dec(bct, bst), "none", None, None, F32)
    assert dct.shape == (N, 320) and xct.shape == (C, 320)
    db = fos.linear8(dct, dst, xct, xst, out_dtype=F32)
    _check(db, None, dec(dct, dst), dec(xct, xst), "none", None, None, F32)


def test_empty_tokens():
    b, _ = _operand(8, _rand(64, 128, 1))
    e = torch.empty(0, 128, dtype=torch.uint8, device=DEV)
    out = fos.linear8(e, torch.empty(0, dtype=torch.uint8, device=DEV), b[0], b[1])
    assert out.shape == (0, 64)


def test_refusals():
    a, _ = _operand(8, _rand(8, 128, 1))
    b, _ = _operand(8, _rand(64, 128, 2))
    for args, kw, err in [
        ((a[0].cpu(), a[1], b[0], b[1]), {}, ValueError),
        ((a[0], a[1][:-1], b[0], b[1]), {}, ValueError),
        ((a[0], a[1].float(), b[0], b[1]), {}, ValueError),
        ((a[0], a[1], b[0][:, :64].contiguous(), b[1]), {}, ValueError),
        ((a[0], a[1], b[0], b[1]), dict(act="tanh"), ValueError),
        ((a[0], a[1], b[0], b[1]), dict(bias=torch.ones(63, device=DEV)), ValueError),
        ((a[0], a[1], b[0], b[1]), dict(bias=torch.ones(64, device=DEV).double()), ValueError),
        ((a[0], a[1], b[0], b[1]), dict(residual=torch.ones(8, 64, device=DEV)), ValueError),
        ((a[0], a[1], b[0], b[1]), dict(out=torch.ones(8, 64, device=DEV)), ValueError),
        ((a[0], a[1], b[0], b[1]), dict(out_dtype=torch.float64), ValueError),
    ]:
        with pytest.raises(err):
            fos.linear8(*args, **kw)
    c, s, _, _ = fos.quantize8(_rand(24, 128, 1))
    with pytest.raises(fos.FosError) as e:
        fos.linear8(a[0], a[1], c, s)  # N = 24
    assert e.value.status == fos.FOS_ERR_UNSUPPORTED
    q, _ = _operand(4, _rand(8, 128, 1), True)
    w, _ = _operand(4, _rand(64, 128, 1))
    with pytest.raises(ValueError):
        fos.linear4(*q, *w)  # per-row amax without row_scaled


@pytest.mark.parametrize("fmt", [8, 4])
@pytest.mark.parametrize("M,N,K", [(2500, 4096, 1024), (3000, 2304, 4096), (200, 14336, 2048),
                                   (64, 4096, 4096)])
def test_many_calls_one_answer(fmt, M, N, K):
    """Products of many tiles back to back, other products between them: every
    repeat equals the first bit for bit."""
    a, _ = _operand(fmt, _rand(M, K, 1))
    b, _ = _operand(fmt, _rand(N, K, 2))
    a2, _ = _operand(fmt, _rand(17, K, 3))
    res = _rand(M, N, 4).to(BF16)
    one = _call(fmt, a, b, act="silu", residual=res)
    outs = []
    for _ in range(12):
        _call(fmt, a2, b)
        outs.append(_call(fmt, a, b, act="silu", residual=res))
    for o in outs:
        assert torch.equal(one, o)


def test_outputs_past_2_to_the_31_elements():
    """150,000 x 14,336 outputs (2.15e9): the last rows equal those of a product
    of the last rows alone."""
    M, N, K = 150000, 14336, 128
    x = _rand(M, K, 1)
    a, _ = _operand_codes(x)
    b, _ = _operand_codes(_rand(N, K, 2))
    out = fos.linear8(*a, *b, act="relu", out_dtype=BF16)
    r0 = (M - 300) // 128 * 128
    tail, _ = _operand_codes(x[r0:].contiguous())
    assert torch.equal(out[r0:], fos.linear8(*tail, *b, act="relu", out_dtype=BF16))


def _operand_codes(x):
    c, s, _, _ = fos.quantize8(x)
    return (c, s), None


def test_ffn_block_example():
    """The example's training step and decode step: results of 8-bit operands
    are within a few hundredths of the unquantized block's (an E4M3 operand is
    off by 2^-5 at most, 0.02 to 0.03 on average; NVFP4 by about 0.1)."""
    import importlib.util
    import os
    p = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "ffn_block.py")
    spec = importlib.util.spec_from_file_location("ffn_block", p)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    for act, tokens in (("gelu_tanh", 333), ("silu", 64)):
        err = m.run(tokens, 512, 1536, act)
        for k, v in err.items():
            assert v < (0.3 if "NVFP4" in k else 0.1), (act, k, v)
