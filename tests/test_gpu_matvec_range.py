"""matvec4 takes every element of x as it is, whatever stands beside it and whatever
the weights' decode scale: rows whose large elements meet zero weights, so that a
result is of the small ones alone, and weights and rows far from 1, against 64 bits.

Bounds, e = 2^-24, K terms: 2 (K + 16) e sum |x w| as in test_gpu_experts.py, of the terms
that a result has.  For results of one term: the weight and its decode scale are
exact up to the one rounding that the reference has too; three products with the
scale and sums of three pieces are six roundings, and subnormal results round by
half of 2^-149 as often.
"""
import pytest
import torch

import expert_reference as ex
import nvfp4_quantization_precision_gb300 as fos

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = torch.float64
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
CFG = fos.Config(scale_tiled=True)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _rand(*shape, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV)


def _uniform(lo, hi, *shape, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return lo + (hi - lo) * torch.rand(*shape, generator=g, device=DEV)


def _weights(w):
    """NVFP4 weights and their exact values with the decode scale."""
    N, K = w.shape
    c, s, a = fos.quantize(w.to(BF16), CFG)
    return (c, s, a), ex.values4(c, ex.untile(s, N, K // 16)) * ex.decode_scale(a)


def _check(x, b, wv, ids=None, bound=None):
    """Every result within the bound of its own terms."""
    got = fos.matvec4(x, *b, ids=ids, out_dtype=F32).to(D)
    xd = x.to(D)
    want = xd @ wv.t()
    K = x.shape[1]
    err = (xd.abs() @ wv.abs().t()) * (2.0 * (K + 16) * 2.0 ** -24) + 2.0 ** -149 * (K / 16 + 8)
    off = (got - want).abs() - err
    assert torch.isfinite(got).all()
    assert (off <= 0).all(), float(off.max())


def _magnitudes(x, lo, hi, seed):
    """x with magnitudes spread over 2^lo .. 2^hi."""
    return torch.ldexp(x, torch.floor(_uniform(lo, hi, *x.shape, seed=seed)).int()).float()


def _bands(x, N, width, lo):
    """Weights N x K: row n meets the elements of x's first row with magnitudes in a band of
    `width` binades, and zeros elsewhere."""
    e = torch.log2(x[0].abs().to(D))
    w = _rand(N, x.shape[1], seed=5)
    w = w + 0.5 * w.sign()
    for n in range(N):
        at = lo + width * n
        w[n] *= (e >= at) & (e < at + width)
    return w


# K of one step, with an end inside one, of several parts of x (above 2048 for eight rows)
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("M,K", [(1, 128), (1, 416), (8, 512), (3, 1056), (8, 4128), (11, 2048), (2, 6176)])
def test_small_elements_beside_large_ones(dt, M, K):
    x = _rand(M, K, seed=M)
    x = _magnitudes(x.sign() * (1 + 0.9 * x.abs().clamp(max=1)), -100, 100, K).to(dt)
    w = _bands(x, 16, 12.5, -100)
    b, wv = _weights(w)
    _check(x, b, wv)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_one_element_a_result(dt):
    """A diagonal of weights: each result is one element's product, from subnormal ones to
    2^100, with all of an element's bits."""
    K = 512
    w = 6.0 * torch.eye(K, device=DEV)
    b, wv = _weights(w)
    lo = -132 if dt == BF16 else -148
    x = torch.stack([_magnitudes(1 + _uniform(0, 0.99, K, seed=1), lo, 100, 2),
                     _magnitudes(-1 - _uniform(0, 0.99, K, seed=3), lo, -100, 4),
                     _magnitudes(1 + _uniform(0, 0.99, K, seed=5), -40, 0, 6),
                     _magnitudes(1 + _uniform(0, 0.99, K, seed=7), 60, 100, 8)])
    x[0, ::3] = 0
    x = x.to(dt)
    got = fos.matvec4(x, *b, out_dtype=F32).to(D)
    want = x.to(D) @ wv.t()
    assert ((got - want).abs() <= want.abs() * (6 * 2.0 ** -24) + 6 * 2.0 ** -150).all()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_a_large_element_with_a_zero_weight(dt):
    K, N = 256, 32
    w = _rand(N, K, seed=1)
    w[:, 5] = 0
    w[:, 200] = 0
    b, wv = _weights(w)
    x = _rand(2, K, seed=2)
    x[0, 5], x[0, 200] = 1e12, -3e30
    x[0, 1], x[1, 200] = 1.328, 3e38
    _check(x.to(dt), b, wv)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_tails_of_an_activation(dt):
    """What an activation leaves of large negative arguments."""
    K, N = 4096, 48
    z = 4 * _rand(5, K, seed=1).to(D)
    x = (0.5 * z * torch.special.erfc(-z / 2 ** 0.5)).to(dt)
    small = x[0].abs() < 1e-12
    w = _rand(N, K, seed=2)
    w[: N // 2, ~small] = 0
    assert small.sum() > 20
    b, wv = _weights(w)
    _check(x, b, wv)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_rows_beside_a_wide_one(dt):
    """A row of many magnitudes changes nothing of the others, in no part of K."""
    M, K = (8, 4128) if dt == BF16 else (2, 4128)
    b, wv = _weights(_rand(80, K, seed=1))
    x = _rand(M, K, seed=2).to(dt)
    before = fos.matvec4(x, *b, out_dtype=F32)
    for lo, hi in ((0, 128), (2048, 2176), (4096, 4128), (0, K)):
        y = x.clone()
        y[1, lo:hi] = _magnitudes(_rand(hi - lo, seed=3), -100, 60, 4).to(dt)
        got = fos.matvec4(y, *b, out_dtype=F32)
        assert torch.equal(got[0], before[0]) and torch.equal(got[2:], before[2:])
        _check(y, b, wv)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("N,K", [(16, 8192), (1040, 4096), (4112, 2048), (14336, 1024)])
def test_in_every_launch(dt, N, K):
    """Clusters along K, one to four tiles of rows a CTA."""
    for M in (1, 9):
        x = _magnitudes(_rand(M, K, seed=1), -60, 60, 2).to(dt)
        w = _rand(N, K, seed=3)
        w[:, x[0].abs() > 1] = 0
        b, wv = _weights(w)
        _check(x, b, wv)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_experts_with_rows_of_many_magnitudes(dt):
    K, N, ids = 1056, 144, [1, 0, 1, 1, 2, 1, 1, 1, 1, 1, 1, 1]
    x = _magnitudes(_rand(len(ids), K, seed=1), -80, 80, 2).to(dt)
    w = _rand(3, N, K, seed=3)
    for e in range(3):
        w[e][:, x[e].abs() > 1e-6] = 0
    q = [_weights(w[e]) for e in range(3)]
    b = [torch.stack([v[0][0] for v in q]), torch.stack([v[0][1] for v in q]), torch.cat([v[0][2] for v in q])]
    got = fos.matvec4(x, *b, ids=torch.tensor(ids, dtype=torch.int32, device=DEV), out_dtype=F32).to(D)
    for p, e in enumerate(ids):
        xd, wv = x[p:p + 1].to(D), q[e][1]
        err = (xd.abs() @ wv.abs().t()) * (2.0 * (K + 16) * 2.0 ** -24) + 2.0 ** -140
        assert ((got[p:p + 1] - xd @ wv.t()).abs() <= err).all()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_infinities_beside_many_magnitudes(dt):
    K, N = 512, 48
    b, wv = _weights(_rand(N, K, seed=1))
    x = _magnitudes(_rand(3, K, seed=2), -90, 90, 3).to(dt)
    clean = fos.matvec4(x, *b, out_dtype=F32)
    x[1, 7], x[2, 9] = float("inf"), float("nan")
    got = fos.matvec4(x, *b, out_dtype=F32)
    assert torch.equal(got[0], clean[0]) and torch.isnan(got[2]).all()
    w7 = wv[:, 7]
    assert torch.isnan(got[1][w7 == 0]).all()
    assert (got[1][w7 > 0] == float("inf")).all() and (got[1][w7 < 0] == float("-inf")).all()


def test_repeats_with_rows_of_many_magnitudes():
    K, N = 7168, 2048
    b, _ = _weights(_rand(N, K, seed=1))
    x = _magnitudes(_rand(8, K, seed=2), -60, 60, 3).to(BF16)
    one = fos.matvec4(x, *b, out_dtype=F32)
    outs = [fos.matvec4(x, *b, out_dtype=F32) for _ in range(40)]
    assert all(torch.equal(one, o) for o in outs)


def _scaled_weights(N, K, size, seed):
    """Weights of magnitudes around `size`, as whole parts of it, and their exact values."""
    w = (_rand(N, K, seed=seed).to(BF16).to(D) * size).to(F32)
    c, s, a = fos.quantize(w, CFG)
    S = torch.clamp(torch.tensor(2688.0) / a.cpu(), max=torch.finfo(F32).max)
    return (c, s, a), ex.values4(c, ex.untile(s, N, K // 16)) * (1 / S).to(D).to(DEV)


# the decode scale and x far from 1 in either direction, their product in range
@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("weights,size", [(1e35, 1.0), (1e35, 1e-4), (2e36, 0.5), (1e30, 100.0), (1e-35, 1.0), (1e-30, 1e-3),
                                          (1e-38, 1e4), (1e-35, 1e36), (1e-38, 1e37), (1e35, 1e-36), (1e35, 1e-38),
                                          (1e10, 1e-40), (1e-20, 1e-15)])
def test_scales_of_the_weights(dt, weights, size):
    if dt == F16 and not 1e-4 <= size <= 1e4:
        size = 1.0
    K, N = 544, 48
    b, wv = _scaled_weights(N, K, weights, 1)
    _check((_rand(3, K, seed=2) * size).to(dt), b, wv)
    if dt != F16:
        x = _magnitudes(_rand(3, K, seed=3), -40, 0, 4) * size
        _check(x.to(dt), b, wv)
