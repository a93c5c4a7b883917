"""Plain 64-bit forms of the operators on rows packed by expert, used by their tests.
Nothing here calls the library; formats are those of ffn_reference."""
import torch

import ffn_reference as ref

D = torch.float64


def ends(offs, rows):
    """Clamped cumulative ends."""
    out, e = [], 0
    for o in offs:
        e = max(e, min(rows, max(e, int(o))))
        out.append(e)
    return out


def spans(offs, rows):
    """(expert, first row, end, first padded column, padded end)."""
    out, r, p = [], 0, 0
    for g, e in enumerate(ends(offs, rows)):
        q = p + -(-(e - r) // 128) * 128
        out.append((g, r, e, p, q))
        r, p = e, q
    return out


def columns(rows, groups):
    """Most columns that `rows` rows of `groups` experts can take."""
    return (rows + 127 * min(rows, groups)) // 128 * 128


def untile(flat, rows, n):
    """Scale bytes [rows, n] from the tiled layout, where they are."""
    return flat[ref.tile_index(rows, n).to(flat.device)]


def values8(codes, scales):
    """Doubles of E4M3 codes [R, K] and scale bytes [R, K/32]."""
    R, K = codes.shape
    v = codes.view(torch.float8_e4m3fn).to(torch.float32).to(D).view(R, K // 32, 32)
    return (v * ref.pow2(scales.long() - 127).unsqueeze(2)).view(R, K)


def values4(codes, scales):
    """Doubles of E2M1 codes [R, K/2] times their E4M3 scales [R, K/16]."""
    R, K = codes.shape[0], codes.shape[1] * 2
    t = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=D,
                     device=codes.device)
    v = t[torch.stack((codes & 15, codes >> 4), 2).long()].view(R, K // 16, 16)
    return (v * scales.contiguous().view(torch.float8_e4m3fn).to(torch.float32).to(D).unsqueeze(2)).view(R, K)


def decode_scale(amax):
    """rn(1 / S) of NVFP4 amaxes, as doubles."""
    a = amax.cpu()
    S = torch.tensor(2688.0) / a
    return torch.where(a > 0, 1 / S, torch.ones_like(S)).to(D).to(amax.device)
