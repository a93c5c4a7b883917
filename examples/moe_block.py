"""A mixture-of-experts block on quantized products: one training step in the 8-bit
block format, a batch served with NVFP4 operands, and single tokens served with
NVFP4 weights and tokens that are not quantized.

    h   = x + residual,  z = rms_norm(h) * g
    p   = the top_k of softmax(z . Wr^T),  tokens packed by their expert
    y   = act(z[packed] . Wup[e]^T + b[e]) . Wdown[e]^T
    out = h + sum over a token's experts of p * y

The training step returns out and the gradients of Wup, b, Wdown and of the packed
tokens.  Router, packing and combination are plain torch; every product over the
experts is one call.

    python examples/moe_block.py [--tokens 1000] [--width 1024] [--hidden 2048] [--experts 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_quantization_precision_gb300 as fos  # noqa: E402


class Experts:
    """Weights [G, N, K] of the experts (N and K multiples of 128) in the forms of a
    training framework: 8-bit rows for z . W^T and columns for the input gradient, and
    NVFP4 for serving."""

    def __init__(self, w):
        G, N, K = w.shape
        self.w = w
        # with whole tiles of 128 rows one call quantizes all experts
        c, s = fos.quantize8(w.view(G * N, K))[:2]
        self.rows = c.view(G, N, K), s
        t = [fos.quantize8(e, rowwise=False, colwise=True)[2:] for e in w]
        self.cols = torch.stack([a for a, _ in t]), torch.stack([b for _, b in t])
        q = [fos.quantize(e, fos.Config(scale_tiled=True)) for e in w]
        self.nvfp4 = [torch.stack([e[0] for e in q]), torch.stack([e[1] for e in q]), torch.cat([e[2] for e in q])]


def route(z, wr, top_k):
    """Each token's experts and their weights; the packed order and the experts' ends."""
    p, expert = torch.softmax(z.float() @ wr.float().t(), 1).topk(top_k, 1)
    order = expert.flatten().argsort(stable=True)
    ends = torch.bincount(expert.flatten(), minlength=wr.shape[0]).cumsum(0).to(torch.int32)
    return expert, p / p.sum(1, keepdim=True), order, ends


def forward(z, up, b, down, order, ends, top_k, act="silu"):
    """The experts' outputs for the packed tokens, and what the backward pass reads."""
    packed = z[order // top_k].contiguous()
    zc, zs, zct, zst = fos.quantize8_grouped(packed, ends)
    a, pre = fos.linear8_grouped(zc, zs, *up.rows, ends, act=act, bias=b, out_dtype=z.dtype, save_pre=True)
    ac, as_, act_, ast = fos.quantize8_grouped(a, ends)
    y = fos.linear8_grouped(ac, as_, *down.rows, ends, out_dtype=z.dtype)
    return y, (pre, (act_, ast), (zct, zst))


def backward(dy, saved, up, down, ends, act="silu"):
    """Gradients of the packed tokens, Wup, b and Wdown (the last three fp32)."""
    pre, a_cols, z_cols = saved
    rows, dt = dy.shape[0], dy.dtype
    yc, ys, yct, yst = fos.quantize8_grouped(dy, ends)
    da = fos.linear8_grouped(yc, ys, *down.cols, ends, out_dtype=dt)
    ddown = fos.linear8_grouped_wgrad(yct, yst, *a_cols, ends, rows)
    dc, ds, dct, dst, _, db = fos.act_backward_grouped(da, pre, act, ends)
    dz = fos.linear8_grouped(dc, ds, *up.cols, ends, out_dtype=dt)
    dup = fos.linear8_grouped_wgrad(dct, dst, *z_cols, ends, rows)
    return dz, dup, db, ddown


def serve_batch(z, up, b, down, order, ends, top_k, act="silu"):
    """The experts' outputs for packed tokens with NVFP4 operands."""
    packed = z[order // top_k].contiguous()
    a = fos.linear4_grouped(*fos.quantize_grouped(packed, ends), *up.nvfp4, ends, act=act, bias=b, out_dtype=z.dtype)
    return fos.linear4_grouped(*fos.quantize_grouped(a, ends), *down.nvfp4, ends, out_dtype=z.dtype)


def serve_tokens(z, up, b, down, expert, act="silu"):
    """The experts' outputs for a few tokens, row t * top_k + j of token t's j-th expert."""
    ids = expert.flatten().to(torch.int32)
    a = fos.matvec4(z, *up.nvfp4, ids=ids, act=act, bias=b)
    return fos.matvec4(a, *down.nvfp4, ids=ids)


def combine(h, y, p):
    """h + the experts' outputs (row t * top_k + j) by their weights."""
    return (h.float() + (y.float().view(*p.shape, -1) * p.unsqueeze(2)).sum(1)).to(h.dtype)


def unpack(y, order):
    out = torch.empty_like(y)
    out[order] = y
    return out


def exact(z, wup, b, wdown, expert, dy, act):
    """Outputs per token and expert, and the gradients, unquantized in 64 bits; dy in
    the same order."""
    T, k = expert.shape
    leaves = [t.double().requires_grad_() for t in (z, wup, b, wdown)]
    zz, u, bb, d = leaves
    f = {"silu": torch.nn.functional.silu, "relu": torch.relu, "gelu": torch.nn.functional.gelu}[act]
    rows = zz.unsqueeze(1).expand(T, k, z.shape[1]).reshape(T * k, -1)
    e = expert.flatten()
    y = torch.stack([d[g] @ f(u[g] @ r + bb[g]) for r, g in zip(rows, e.tolist())])
    return y.detach(), torch.autograd.grad((y * dy.double()).sum(), leaves)


def run(tokens=1000, width=1024, hidden=2048, experts=8, top_k=2, act="silu", dtype=torch.bfloat16, seed=0):
    """One training step, one served batch, and four served tokens; relative errors
    against 64 bits without quantization."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    x, residual = rand(tokens, width).to(dtype), rand(tokens, width).to(dtype)
    g, wr = 1 + 0.1 * rand(width), rand(experts, width) * width ** -0.5
    wup = (rand(experts, hidden, width) * width ** -0.5).to(dtype)
    wdown = (rand(experts, width, hidden) * hidden ** -0.5).to(dtype)
    b = 0.1 * rand(experts, hidden)
    up, down = Experts(wup), Experts(wdown)
    _, _, z, h, _ = fos.rms_norm(x, g, residual=residual, quantized=False, normalized=True)
    expert, p, order, ends = route(z, wr, top_k)
    y, saved = forward(z, up, b, down, order, ends, top_k, act)
    out = combine(h, unpack(y, order), p)
    dout = rand(tokens, width).to(dtype)
    # of out to the experts' outputs, in their order
    dy = (dout.float().unsqueeze(1) * p.unsqueeze(2)).to(dtype).view(tokens * top_k, width)
    grads = backward(dy[order].contiguous(), saved, up, down, ends, act)
    want, (wz, wgup, wb, wgdown) = exact(z, wup, b, wdown, expert, dy, act)
    far = lambda a, q: float((a.double() - q).norm() / q.norm())  # noqa: E731
    dz = unpack(grads[0], order).double().view(tokens, top_k, width).sum(1)
    err = {"y": far(unpack(y, order), want), "out": far(out, combine(h.double(), want, p.double())),
           "dz": far(dz, wz), "dup": far(grads[1], wgup), "db": far(grads[2], wb), "ddown": far(grads[3], wgdown)}
    err["batch (NVFP4)"] = far(unpack(serve_batch(z, up, b, down, order, ends, top_k, act), order), want)
    few = min(4, tokens)
    err["tokens (NVFP4 weights)"] = far(serve_tokens(z[:few], up, b, down, expert[:few], act), want[:few * top_k])
    return err


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=1000)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--act", default="silu", choices=("relu", "gelu", "silu"))
    a = ap.parse_args()
    for k, v in run(a.tokens, a.width, a.hidden, a.experts, act=a.act).items():
        print("%-24s relative error %.3g" % (k, v))
