"""The pair kernel of linear8 / linear4 over many chunks of scales: every element
against the product of the decoded operands, at sizes where scale warps wait long
for a buffer in tensor memory while the shared-memory slot they have read is filled
again.  Half of the rows' neighbouring blocks have different scales (standard
deviation 0.05: the largest of 32 magnitudes lies about evenly on both sides of a
power of two's threshold), so a row that took another chunk's scales shows.

Bound of an element, K terms with fp32 accumulation in any order: (K + 4) 2^-24 sum
|a b|; the compared product adds as much.
"""
import pytest
import torch

import ffn_reference as ref
import nvfp4_quantization_precision_gb300 as fos

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _tile(flat, rows, n):
    return flat[ref.tile_index(rows, n).to(DEV)]


def _operand(fmt, rows, K, std, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(rows, K, generator=g, device=DEV) * std
    if fmt == 8:
        c, s, _, _ = fos.quantize8(x)
        two = (_tile(s, rows, K // 32).int() << 23).view(torch.float32)
        v = c.view(torch.float8_e4m3fn).float().view(rows, K // 32, 32) * two.unsqueeze(2)
        return (c, s), v.view(rows, K)
    c, s, a = fos.quantize(x.bfloat16(), fos.Config(scale_tiled=True))
    t = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    v = t[torch.stack((c & 15, c >> 4), 2).long()].view(rows, K // 16, 16)
    v = v * _tile(s, rows, K // 16).view(torch.float8_e4m3fn).float().unsqueeze(2)
    return (c, s, a), v.view(rows, K) * (a / 2688.0)


@pytest.mark.parametrize("fmt,M,N,K", [(8, 8192, 14336, 4096), (8, 14336, 4096, 1024),
                                       (8, 2048, 4096, 7168), (4, 4096, 4096, 14336)])
def test_every_element(fmt, M, N, K):
    a, av = _operand(fmt, M, K, 0.05, 1)
    b, bv = _operand(fmt, N, K, 1.0, 2)
    want = av @ bv.t()
    bound = (av.abs() @ bv.abs().t()) * (2 * (K + 4) * 2.0 ** -24)
    for _ in range(3):
        got = (fos.linear8 if fmt == 8 else fos.linear4)(*a, *b, out_dtype=torch.float32)
        assert ((got - want).abs() <= bound).all(), "elements off: %d" % ((got - want).abs() > bound).sum()
