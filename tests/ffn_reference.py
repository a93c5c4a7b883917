"""Plain 64-bit forms of the feed-forward operators, used by their tests.

Nothing here calls the library: codes and scales are decoded and formed from
the definition of the 8-bit block format (E4M3 codes, one power-of-two scale
per 32 elements), NVFP4 values from their E2M1 table, and the tiled scale
layout is read index by index.
"""
import math

import torch

D = torch.float64
# unit roundoff of the storage types (half a unit in the last place, relative)
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def pow2(e):
    """2^e (integer tensor, normal range) as doubles, from their bits."""
    return ((e.long() + 1023) << 52).view(D)


def tile_index(rows, n):
    """Byte index of scale (r, j) in the tiled layout of a [rows, n] scale matrix."""
    r = torch.arange(rows).unsqueeze(1)
    j = torch.arange(n).unsqueeze(0)
    nc = -(-n // 4)
    return (r // 128 * nc + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4


def untile(flat, rows, n):
    return flat.cpu()[tile_index(rows, n)]


def padding(flat, rows, n):
    """The bytes of a tiled buffer that belong to no scale."""
    keep = torch.ones(flat.numel(), dtype=torch.bool)
    keep[tile_index(rows, n).reshape(-1)] = False
    return flat.cpu()[keep]


def e4m3(codes):
    c = codes.cpu().long()
    ex, man = c >> 3 & 15, (c & 7).to(D)
    v = torch.where(ex > 0, (1 + man / 8) * pow2(ex - 7), man / 512)
    v = torch.where((c & 127) == 127, torch.full_like(v, math.nan), v)
    return torch.where(c >> 7 > 0, -v, v)


def scale_of(amax):
    """Scale byte from the exact rule: smallest e >= -127 with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax / 448.0)
    e = torch.where(m > 0.5, e, e - 1)
    e = torch.where(amax == 0, torch.full_like(e, -127), e).clamp(min=-127)
    return torch.where(torch.isinf(amax), torch.full_like(e, 120), e) + 127


def blocks(v):
    return v.reshape(v.shape[0], -1, 32)


def amax_of(v):
    return torch.nan_to_num(blocks(v).abs(), nan=0.0, posinf=math.inf).amax(2)


def quantize8(v):
    """(code values, scale bytes) of the exact values v [R, C] in doubles."""
    s = scale_of(amax_of(v))
    y = blocks(v) * pow2(127 - s).unsqueeze(2)
    _, k = torch.frexp(y)
    k = (k - 4).clamp(min=-9)
    q = (torch.round(y * pow2(-k)) * pow2(k)).clamp(-448, 448)
    return q.reshape(v.shape), s


def check_codes(codes, scales, v, rel):
    """codes / scale bytes [R, C/32] against exact values v, of which the
    kernel's own values may be off by the relative bound `rel` [like v, or a
    number] of the element: a scale byte may differ only where the block's
    largest value is that close to its threshold, and a code must be within
    half an E4M3 step (plus that bound) of the value under its scale."""
    v = v.cpu()
    rel = rel.cpu() if isinstance(rel, torch.Tensor) else torch.full_like(v, rel)
    s = scales.cpu().long()
    a = amax_of(v)
    r = amax_of(rel * 0 + rel) if rel.numel() else a
    lo, hi = scale_of(a * (1 - r)), scale_of(a * (1 + r))
    assert ((s >= lo) & (s <= hi)).all(), "scale bytes"
    y = blocks(v) * pow2(127 - s).unsqueeze(2)
    got = blocks(e4m3(codes))
    nan = torch.isnan(y)
    assert torch.equal(nan, torch.isnan(got)), "NaN codes"
    _, k = torch.frexp(torch.nan_to_num(y, nan=0.0, posinf=448.0, neginf=-448.0))
    half = pow2((k - 5).clamp(min=-10))
    want = y.clamp(-448, 448)
    err = (got - want).abs()
    bad = ~nan & (err > half * (1 + 1e-12) + blocks(rel) * want.abs())
    assert not bad.any(), "codes: %d off, worst %g steps" % (bad.sum(), (err / half)[~nan].max())


def near(got, want, bound, what):
    """|got - want| <= bound element by element; non-finite values equal."""
    got, want = got.to(D).cpu(), want.cpu()
    bound = bound.cpu() if isinstance(bound, torch.Tensor) else torch.full_like(want, bound)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(want), torch.isnan(got)), what + ": NaN places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what + ": infinities"
    over = (got - want).abs()[fin] > bound[fin]
    assert not over.any(), "%s: %d over the bound, worst ratio %g" % (
        what, over.sum(), ((got - want).abs()[fin] / bound[fin].clamp(min=1e-300)).max())


def act(v, name):
    if name == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if name == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if name == "silu":
        return v * torch.sigmoid(v)
    return v


def act_slope(p, name):
    """The derivative in closed form."""
    if name == "relu":
        return (p > 0).to(D)
    if name == "gelu":
        return 0.5 * torch.erfc(-p / math.sqrt(2)) + p * torch.exp(-p * p / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (p + 0.044715 * p ** 3))
        return 0.5 * (1 + t) + 0.5 * p * (1 - t * t) * c * (1 + 3 * 0.044715 * p * p)
    if name == "silu":
        s = torch.sigmoid(p)
        return s * (1 + p * (1 - s))
    return torch.ones_like(p)
