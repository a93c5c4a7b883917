"""A feed-forward block on quantized products: one training step in the 8-bit
block format, and the same block serving single tokens with NVFP4 weights.

    h   = x + residual
    z   = rms_norm(h) * g                     8-bit rows and columns
    a   = act(z . Wup^T + b)                  pre-activation kept
    out = a . Wdown^T + h

The training step returns out, the gradients of x (and the residual), g, Wup, b
and Wdown.  Every product runs on operands in 8 bits: the weights and the
activations are quantized along their rows for the forward products and along
their columns for the gradients', as a training framework would keep them.

    python examples/ffn_block.py [--tokens 1000] [--width 1024] [--hidden 4096]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_quantization_precision_gb300 as fos  # noqa: E402


class Weights:
    """A weight [N, K] with its 8-bit forms: rows for x . W^T, columns for the
    input gradient dy . W."""

    def __init__(self, w):
        self.w = w
        self.rows = fos.quantize8(w)[:2]
        self.cols = fos.quantize8(w, rowwise=False, colwise=True)[2:]


def forward(x, residual, g, up, b, down, act="gelu_tanh"):
    """Block output and what the backward pass reads."""
    zc, zs, z, h, rstd = fos.rms_norm(x, g, residual=residual, normalized=True)
    a, pre = fos.linear8(zc, zs, *up.rows, act=act, bias=b, out_dtype=x.dtype, save_pre=True)
    # a along its rows for the down projection, z and a along their columns for
    # the weight gradients
    ac, as_, act_, ast = fos.quantize8(a, colwise=True)
    zct, zst = fos.quantize8(z, rowwise=False, colwise=True)[2:]
    out = fos.linear8(ac, as_, *down.rows, residual=h, out_dtype=x.dtype)
    return out, (h, rstd, pre, (act_, ast), (zct, zst))


def backward(dout, saved, g, up, down, act="gelu_tanh"):
    """Gradients of x (the residual's is the same), g, Wup, b, Wdown (fp32)."""
    h, rstd, pre, a_cols, z_cols = saved
    dt = dout.dtype
    # dout is also the gradient that reaches h past the block
    oc, os_, oct_, ost = fos.quantize8(dout, colwise=True)
    da = fos.linear8(oc, os_, *down.cols, out_dtype=dt)
    ddown = fos.linear8(oct_, ost, *a_cols, out_dtype=torch.float32)
    pc, ps, pct, pst, _, db = fos.act_backward(da, pre, act)
    dz = fos.linear8(pc, ps, *up.cols, out_dtype=dt)
    dup = fos.linear8(pct, pst, *z_cols, out_dtype=torch.float32)
    dx, dg = fos.rms_norm_backward(dz, h, rstd, g, dh=dout)
    return dx, dg, dup, db, ddown


def serve(x, residual, g, up4, b, down4, act="gelu_tanh"):
    """One decode step with NVFP4 weights (codes, tiled scales, amax)."""
    cfg = fos.Config(row_scaled=True, scale_tiled=True)
    _, _, z, h, _ = fos.rms_norm(x, g, residual=residual, quantized=False, normalized=True)
    a = fos.linear4(*fos.quantize(z, cfg), *up4, act=act, bias=b, out_dtype=x.dtype, cfg=cfg)
    return fos.linear4(*fos.quantize(a, cfg), *down4, residual=h, out_dtype=x.dtype, cfg=cfg)


def exact(x, residual, g, wup, b, wdown, dout, act):
    """The block and its gradients with unquantized operands, in 64 bits."""
    leaves = [t.double().requires_grad_() for t in (x, g, wup, b, wdown)]
    xx, gg, u, bb, d = leaves
    h = xx + residual.double()
    z = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * gg
    p = z @ u.t() + bb
    a = {"gelu": lambda v: torch.nn.functional.gelu(v),
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh"),
         "silu": torch.nn.functional.silu, "relu": torch.relu}[act](p)
    out = a @ d.t() + h
    return out.detach(), torch.autograd.grad((out * dout.double()).sum(), leaves)


def run(tokens=1000, width=1024, hidden=4096, act="gelu_tanh", dtype=torch.bfloat16, seed=0):
    """One training step and one decode step; relative errors of every result
    against 64 bits without quantization."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    x, residual = rand(tokens, width).to(dtype), rand(tokens, width).to(dtype)
    g, b = 1 + 0.1 * rand(width), 0.1 * rand(hidden)
    wup, wdown = (rand(hidden, width) * width ** -0.5).to(dtype), (rand(width, hidden) * hidden ** -0.5).to(dtype)
    dout = rand(tokens, width).to(dtype)
    up, down = Weights(wup), Weights(wdown)
    out, saved = forward(x, residual, g, up, b, down, act)
    grads = backward(dout, saved, g, up, down, act)
    want, wgrads = exact(x, residual, g, wup, b, wdown, dout, act)
    far = lambda p, q: float((p.double() - q).norm() / q.norm())  # noqa: E731
    err = {"out": far(out, want)}
    for name, p, q in zip(("dx", "dg", "dup", "db", "ddown"), grads, wgrads):
        err[name] = far(p, q)
    tiled = fos.Config(scale_tiled=True)
    up4, down4 = fos.quantize(wup, tiled), fos.quantize(wdown, tiled)
    token = serve(x[:1], residual[:1], g, up4, b, down4, act)
    err["token (NVFP4)"] = far(token, want[:1])
    return err


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=1000)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--act", default="gelu_tanh", choices=("relu", "gelu", "gelu_tanh", "silu"))
    a = ap.parse_args()
    for k, v in run(a.tokens, a.width, a.hidden, a.act).items():
        print("%-14s relative error %.3g" % (k, v))
