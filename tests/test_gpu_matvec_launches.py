"""Every launch of matvec4 against 64 bits: one to four tiles of 16 weight rows a CTA, one to
eight CTAs along K, x in one part of shared memory and in several (from 17 steps of
K a CTA on for eight rows, or for two of fp32), for every type of x, one matrix and
experts.  Bound as in test_gpu_experts.py: 2 (K + 16) 2^-24 sum |x w|, then one
rounding each for the bias and the residual, and the result's type."""
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


def _run(M, N, K, dt, G=0, ids=None, X=None):
    X = M if X is None else X
    cfg = fos.Config(scale_tiled=True)
    q, wv = [], []
    for e in range(max(G, 1)):
        c, s, a = fos.quantize(_rand(N, K, seed=e).to(BF16), cfg)
        q.append((c, s, a))
        wv.append(ex.values4(c, ex.untile(s, N, K // 16)) * ex.decode_scale(a))
    x = _rand(X, K, seed=20).to(dt)
    bias, res = _rand(max(G, 1), N, seed=21), _rand(M, N, seed=22).to(dt)
    if G:
        b = [torch.stack([t[0] for t in q]), torch.stack([t[1] for t in q]), torch.cat([t[2] for t in q])]
        got = fos.matvec4(x, *b, ids=torch.tensor(ids, dtype=torch.int32, device=DEV), bias=bias, residual=res)
    else:
        ids = [0] * M
        got = fos.matvec4(x, *q[0], bias=bias[0], residual=res)
    xd = x.to(D)
    for e in set(ids):
        p = [i for i in range(M) if ids[i] == e]
        rows = [i // (M // X) for i in p]
        v = xd[rows] @ wv[e].t()
        err = (xd[rows].abs() @ wv[e].abs().t()) * (2.0 * (K + 16) * 2.0 ** -24)
        v = v + bias[e].to(D)
        err = err + v.abs() * 2.0 ** -23
        out = v + res[p].to(D)
        err = err + out.abs() * 2.0 ** -23
        ref.near(got[p], out, err * 1.01 + out.abs() * ref.U[dt] * (1 + 2.0 ** -10) + ref.TINY[dt], "out")


# rows, N, K                                              tiles, CTAs of a cluster
SIXTEEN = [(1, 16, 32), (1, 16, 4096), (1, 16, 8192),           # 1: 1, 4, 8
           (9, 4112, 32), (9, 2064, 14336), (9, 1040, 4096), (9, 528, 8192),    # 2: 1, 2, 4, 8
           (9, 6160, 32), (1, 6160, 4096),                      # 3: 1, 2
           (9, 8208, 32), (9, 4112, 14336), (9, 2064, 16384), (9, 1040, 8192),  # 4: 1, 2, 4, 8
           (8, 8208, 4128), (11, 14336, 2176), (16, 16400, 2080)]               # parts of x
THIRTY_TWO = [(1, 16, 32), (1, 16, 4096), (1, 16, 8192),
              (9, 1040, 32), (8, 1040, 14336), (9, 272, 4096), (9, 144, 8192),
              (9, 2064, 32), (9, 1040, 4096), (9, 528, 6176), (9, 272, 8192),
              (8, 4112, 32), (8, 2064, 14336), (8, 1040, 16384), (8, 528, 8192),
              (2, 16400, 4128), (5, 8208, 2208)]


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("M,N,K", SIXTEEN)
def test_one_matrix(dt, M, N, K):
    _run(M, N, K, dt)


@pytest.mark.parametrize("M,N,K", THIRTY_TWO)
def test_one_matrix_fp32(M, N, K):
    _run(M, N, K, F32)


# experts named by as many rows at least
@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("G,N,K", [(2, 16, 32), (8, 272, 14336), (2, 16, 4096), (2, 16, 8192),
                                   (2, 4112, 32), (2, 2064, 14336), (2, 1040, 4096), (2, 528, 8192),
                                   (2, 6160, 32), (4, 2064, 4096), (4, 1040, 6176), (4, 528, 8192),
                                   (2, 8208, 32), (2, 4112, 14336), (2, 2064, 16384), (2, 1040, 8192),
                                   (8, 4096, 4128)])
def test_experts(dt, G, N, K):
    r = random.Random(N + K)
    ids = list(range(G)) + [r.randrange(G) for _ in range(G)]
    r.shuffle(ids)
    _run(2 * G, N, K, dt, G, ids)
    ids = ids[:G] if len(set(ids[:G])) > 1 else list(range(G))
    _run(G, N, K, dt, G, ids, X=G // 2)


@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_many_rows_of_an_expert_in_parts(dt):
    """Chunks of eight rows (two of fp32), each through several parts of x."""
    _run(19, 2064, 4128, dt, 2, [1] * 11 + [0] + [1] * 7)


# three tiles, clusters of 2, 4 and 8
@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("N,K", [(2064, 4096), (1040, 6176), (528, 8192)])
def test_three_of_four_experts(dt, N, K):
    _run(3, N, K, dt, 4, [2, 0, 3])
