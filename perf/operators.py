"""Measured cases of the feed-forward block's operators around the quantized products.

Four operators, each in its plain form (elementary torch operations in 32 bits)
and, with ``own`` true, through the package's entry points:

  norm       rms_norm: h = x + residual, its root-mean-square norm times a
             weight, written as E4M3 codes with one power-of-two scale per 32
             elements of a row, next to h and the rows' 1/rms
  norm_back  rms_norm_backward: the gradients of x (or of the residual, they
             are the same) and of the weight
  quant      quantize8 and act_backward: a tensor, or the gradient of an
             activation, written in 8 bits along its rows and along its
             columns, with the bias gradient
  linear     linear8 and linear4: act(a . b^T + bias) + residual from operands
             in 8 bits (32-element blocks) or in NVFP4 (16-element blocks)

Scales are in the tiled layout of block-scaled products (128 x 4 tiles of 512
bytes) unless a case says plain.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token through the norm before the up projection: latency
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "dt": "bf16",
         "residual": True, "tiled": True},
        # an odd decode batch, no residual (the first norm of a stack), plain scales
        {"name": "norm_batch_odd", "op": "norm", "rows": 333, "cols": 2048, "dt": "f16",
         "residual": False, "tiled": False},
        # a training or prefill step's tokens through a wide model's norm
        {"name": "norm_prefill", "op": "norm", "rows": 16384, "cols": 7168, "dt": "bf16",
         "residual": True, "tiled": True},
        # the norm's backward in training, with the residual stream's gradient
        {"name": "norm_back_train", "op": "norm_back", "rows": 8192, "cols": 4096, "dt": "bf16",
         "dh": True},
        # the same in 32 bits over an odd number of rows, no residual branch
        {"name": "norm_back_odd", "op": "norm_back", "rows": 1021, "cols": 7168, "dt": "f32",
         "dh": False},
        # a weight quantized for the forward product and, transposed, for the input gradient
        {"name": "quant_weight", "op": "quant", "rows": 14336, "cols": 4096, "dt": "bf16",
         "act": "none", "bias": False, "value": False, "tiled": True},
        # the gradient behind the up projection's activation, in both directions, with dbias
        {"name": "quant_act_grad", "op": "quant", "rows": 8192, "cols": 14336, "dt": "bf16",
         "act": "silu", "bias": True, "value": False, "tiled": True},
        # the same for a ragged micro-batch in fp16, the gradient itself kept too
        {"name": "quant_act_odd", "op": "quant", "rows": 1000, "cols": 2048, "dt": "f16",
         "act": "gelu", "bias": True, "value": True, "tiled": True},
        # up projection of one token
        {"name": "linear8_token", "op": "linear", "fmt": 8, "M": 1, "N": 14336, "K": 4096,
         "act": "silu", "bias": True, "residual": False, "pre": False, "row": False,
         "dt": "bf16"},
        # down projection of a decode batch, NVFP4, added to the residual stream
        {"name": "linear4_batch", "op": "linear", "fmt": 4, "M": 48, "N": 4096, "K": 14336,
         "act": "none", "bias": False, "residual": True, "pre": False, "row": True,
         "dt": "bf16"},
        # up projection of a training step, pre-activation kept for the backward pass
        {"name": "linear8_train", "op": "linear", "fmt": 8, "M": 8192, "N": 14336, "K": 4096,
         "act": "gelu_tanh", "bias": True, "residual": False, "pre": True, "row": False,
         "dt": "bf16"},
        # down projection of a ragged prefill, NVFP4, everything in the epilogue
        {"name": "linear4_prefill", "op": "linear", "fmt": 4, "M": 5003, "N": 4096, "K": 14336,
         "act": "gelu", "bias": True, "residual": True, "pre": False, "row": True, "dt": "f16"},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(("norm", "norm_back", "quant", "linear"))
    if op == "linear":
        fmt = rng.choice((8, 4))
        while True:
            M, N, K = _log(rng, 1, 8192), _log(rng, 256, 16384, 16), _log(rng, 256, 16384, 32)
            if M * N * K <= 8192 * 14336 * 4096 and M * N <= 8192 * 14336 and 3072 not in (M, N, K):
                break
        return {"op": op, "fmt": fmt, "M": M, "N": N, "K": K, "act": rng.choice(ACTS),
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.5,
                "pre": rng.random() < 0.3, "row": fmt == 4 and rng.random() < 0.5,
                "dt": rng.choice(("bf16", "bf16", "f16", "f32"))}
    most = {"norm": 16384 * 7168, "norm_back": 16384 * 4096, "quant": 8192 * 14336}[op]
    while True:
        rows, cols = _log(rng, 1, 32768), _log(rng, 256, 16384, 32)
        if rows * cols <= most and 3072 not in (rows, cols):
            break
    c = {"op": op, "rows": rows, "cols": cols, "dt": rng.choice(("bf16", "bf16", "f16", "f32"))}
    if c["dt"] == "f32" and rows * cols > most // 2:
        c["dt"] = "bf16"
    if op == "norm":
        c.update(residual=rng.random() < 0.6, tiled=rng.random() < 0.7)
    elif op == "norm_back":
        c.update(dh=rng.random() < 0.6)
    else:
        act = rng.choice(ACTS)
        c.update(act=act, bias=act != "none" and rng.random() < 0.7,
                 value=act != "none" and rng.random() < 0.3, tiled=rng.random() < 0.7)
    return c


# ------------------------------------------------------------------ shared plain pieces
def _tiles(s):
    """[R, n] scale bytes -> flat 128 x 4 tiles of 512 bytes, zero padded."""
    R, n = s.shape
    p = torch.zeros((R + 127) // 128 * 128, (n + 3) // 4 * 4, dtype=torch.uint8, device=s.device)
    p[:R, :n] = s
    return (p.view(p.shape[0] // 128, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
            .reshape(-1).contiguous())


def _untiles(t, R, n):
    r, c = (R + 127) // 128, (n + 3) // 4
    return t.view(r, c, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(r * 128, c * 4)[:R, :n]


def _mx8(v):
    """fp32 [R, C] -> E4M3 codes and UE8M0 scale bytes [R, C/32]: the scale is the smallest
    power of two that keeps the block's largest finite-or-infinite magnitude within 448."""
    R, C = v.shape
    b = v.reshape(R, C // 32, 32)
    a = torch.nan_to_num(b.abs(), nan=0.0, posinf=math.inf).amax(2)
    s = (((a.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp_(0, 254)
    inv = ((254 - s) << 23).view(torch.float32)
    q = (b * inv.unsqueeze(2)).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(R, C), s.to(torch.uint8)


def _held(codes, scales):
    """What codes and scales are held as: E4M3 numbers and powers of two."""
    return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def _act(v, act):
    if act == "relu":
        return v.clamp(min=0.0)
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _act_slope(p, act):
    if act == "relu":
        return (p > 0).to(p.dtype)
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(p * math.sqrt(0.5)))
                + p * torch.exp(-0.5 * p * p) * (1.0 / math.sqrt(2 * math.pi)))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (p + 0.044715 * p * p * p))
        return 0.5 * (1.0 + t) + 0.5 * p * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * p * p)
    s = 1.0 / (1.0 + torch.exp(-p))
    return s * (1.0 + p * (1.0 - s))


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _e2m1_table(dev, dtype=torch.float32):
    return torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=dtype, device=dev)


def _nvfp4(x, row):
    """Standard NVFP4 operand of fp32 x: packed codes, E4M3 scale bytes, amax ([rows] or [1])."""
    R, C = x.shape
    amax = x.abs().amax(1) if row else x.abs().amax().view(1)
    S = (6.0 * 448.0) / amax
    Sr = S.view(-1, 1, 1)
    b = x.view(R, C // 16, 16)
    s8 = ((b.abs().amax(2, keepdim=True) * Sr) / 6.0).to(torch.float8_e4m3fn)
    sig = s8.float()
    y = torch.where(sig > 0, b * (Sr / sig), torch.zeros_like(b))
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    mag = torch.bucketize(y.abs(), edges).to(torch.uint8)
    code = (mag | (torch.signbit(y).to(torch.uint8) << 3)).view(R, C // 2, 2)
    return (code[:, :, 0] | (code[:, :, 1] << 4)).contiguous(), s8.view(torch.uint8).view(R, C // 16), amax


# ------------------------------------------------------------------ inputs
def _acts(g, rows, cols):
    """Activation-like values: N(0, 1) with one entry in a thousand 20 times as large."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    return torch.where(torch.rand(rows, cols, generator=g, device=DEV) < 1e-3, x * 20.0, x)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    dt = DT[case["dt"]]
    s = {"case": case}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        a = _acts(g, M, K)
        b = torch.randn(N, K, generator=g, device=DEV) * 0.02
        if case["fmt"] == 8:
            for n, v in (("a", a), ("b", b)):
                c, sc = _mx8(v)
                s[n], s[n + "s"] = c.view(torch.uint8), _tiles(sc)
        else:
            for n, v, row in (("a", a, case["row"]), ("b", b, False)):
                s[n], sc, s[n + "m"] = _nvfp4(v, row)
                s[n + "s"] = _tiles(sc)
        s["bias"] = (torch.randn(N, generator=g, device=DEV) * 0.5) if case["bias"] else None
        s["residual"] = torch.randn(M, N, generator=g, device=DEV).to(dt) if case["residual"] else None
        s["out"] = torch.empty(M, N, dtype=dt, device=DEV)
        s["pre"] = torch.empty(M, N, dtype=dt, device=DEV) if case["pre"] else None
        return s
    rows, cols = case["rows"], case["cols"]
    u8 = lambda r, c: torch.empty(r, c, dtype=torch.uint8, device=DEV)  # noqa: E731

    def scale_buf(r, n):
        if case["tiled"]:
            return torch.empty((r + 127) // 128 * 128 * ((n + 3) // 4 * 4), dtype=torch.uint8, device=DEV)
        return u8(r, n)

    if case["op"] == "norm":
        s["x"] = _acts(g, rows, cols).to(dt)
        s["residual"] = (torch.randn(rows, cols, generator=g, device=DEV) * 2).to(dt) if case["residual"] else None
        s["weight"] = 1.0 + 0.1 * torch.randn(cols, generator=g, device=DEV)
        s["codes"], s["scales"] = u8(rows, cols), scale_buf(rows, cols // 32)
        s["h"] = torch.empty(rows, cols, dtype=dt, device=DEV) if case["residual"] else None
        s["rstd"] = torch.empty(rows, device=DEV)
    elif case["op"] == "norm_back":
        h = _acts(g, rows, cols).to(dt)
        s["h"] = h
        s["rstd"] = (h.float().square().mean(1) + EPS).rsqrt()
        s["weight"] = 1.0 + 0.1 * torch.randn(cols, generator=g, device=DEV)
        s["dy"] = (torch.randn(rows, cols, generator=g, device=DEV) * 0.05).to(dt)
        s["dh"] = (torch.randn(rows, cols, generator=g, device=DEV) * 0.05).to(dt) if case["dh"] else None
        s["dx"] = torch.empty(rows, cols, dtype=dt, device=DEV)
        s["dweight"] = torch.empty(cols, device=DEV)
    else:
        act = case["act"]
        if act == "none":
            s["x"] = (torch.randn(rows, cols, generator=g, device=DEV) * 0.02).to(dt)
        else:
            s["x"] = (torch.randn(rows, cols, generator=g, device=DEV) * 0.05).to(dt)
            s["pre"] = (torch.randn(rows, cols, generator=g, device=DEV) * 1.5).to(dt)
        pad = (rows + 31) // 32 * 32
        s["codes"], s["scales"] = u8(rows, cols), scale_buf(rows, cols // 32)
        s["codes_t"], s["scales_t"] = u8(cols, pad), scale_buf(cols, pad // 32)
        s["d"] = torch.empty(rows, cols, dtype=dt, device=DEV) if case["value"] else None
        s["dbias"] = torch.empty(cols, device=DEV) if case["bias"] else None
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import nvfp4_quantization_precision_gb300 as fos
    c = s["case"]
    if c["op"] == "norm":
        codes, scales, _, h, rstd = fos.rms_norm(
            s["x"], s["weight"], residual=s["residual"], eps=EPS, scale_tiled=c["tiled"],
            codes=s["codes"], scales=s["scales"], h=s["h"], rstd=s["rstd"])
        codes, scales = _held(codes, scales)
        return {"codes": codes, "scales": scales, "h": h if c["residual"] else None, "rstd": rstd}
    if c["op"] == "norm_back":
        dx, dweight = fos.rms_norm_backward(s["dy"], s["h"], s["rstd"], s["weight"], dh=s["dh"],
                                            dx=s["dx"], dweight=s["dweight"])
        return {"dx": dx, "dweight": dweight}
    if c["op"] == "quant":
        buf = {k: s[k] for k in ("codes", "scales", "codes_t", "scales_t")}
        if c["act"] == "none":
            q = fos.quantize8(s["x"], scale_tiled=c["tiled"], colwise=True, **buf)
            d = dbias = None
        else:
            *q, d, dbias = fos.act_backward(s["x"], s["pre"], c["act"], scale_tiled=c["tiled"],
                                            value=c["value"], bias_grad=c["bias"], d=s["d"],
                                            dbias=s["dbias"], **buf)
        codes, scales = _held(q[0], q[1])
        codes_t, scales_t = _held(q[2], q[3])
        return {"codes": codes, "scales": scales, "codes_t": codes_t, "scales_t": scales_t,
                "d": d, "dbias": dbias}
    more = {"act": c["act"], "bias": s["bias"], "residual": s["residual"], "out": s["out"],
            "pre": s["pre"], "out_dtype": DT[c["dt"]], "save_pre": c["pre"]}
    if c["fmt"] == 8:
        r = fos.linear8(s["a"], s["as"], s["b"], s["bs"], **more)
    else:
        r = fos.linear4(s["a"], s["as"], s["am"], s["b"], s["bs"], s["bm"],
                        cfg=fos.Config(row_scaled=c["row"]), **more)
    return {"out": r[0], "pre": r[1]} if c["pre"] else {"out": r}


def _run_plain(s):
    c = s["case"]
    dt = DT[c["dt"]]
    if c["op"] == "norm":
        h = s["x"].float()
        if c["residual"]:
            h = h + s["residual"].float()
        rstd = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
        codes, sc = _mx8(h * rstd.unsqueeze(1) * s["weight"])
        codes, scales = _held(codes, _tiles(sc) if c["tiled"] else sc)
        return {"codes": codes, "scales": scales, "h": h.to(dt) if c["residual"] else None, "rstd": rstd}
    if c["op"] == "norm_back":
        r = s["rstd"].unsqueeze(1)
        dy, xhat = s["dy"].float(), s["h"].float() * r
        gr = dy * s["weight"]
        dx = (gr - xhat * (gr * xhat).mean(1, keepdim=True)) * r
        if c["dh"]:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(dt), "dweight": (dy * xhat).sum(0)}
    if c["op"] == "quant":
        d = s["x"].float()
        if c["act"] != "none":
            d = d * _act_slope(s["pre"].float(), c["act"])
        codes, sc = _mx8(d)
        t = torch.zeros(c["cols"], (c["rows"] + 31) // 32 * 32, device=d.device)
        t[:, :c["rows"]] = d.t()
        codes_t, sct = _mx8(t)
        codes, scales = _held(codes, _tiles(sc) if c["tiled"] else sc)
        codes_t, scales_t = _held(codes_t, _tiles(sct) if c["tiled"] else sct)
        return {"codes": codes, "scales": scales, "codes_t": codes_t, "scales_t": scales_t,
                "d": d.to(dt) if c["value"] else None, "dbias": d.sum(0) if c["bias"] else None}
    M, N, K = c["M"], c["N"], c["K"]
    if c["fmt"] == 8:
        def deq(q, sc, R):
            two = (_untiles(sc, R, K // 32).int() << 23).view(torch.float32)
            return (q.view(torch.float8_e4m3fn).float().view(R, K // 32, 32) * two.unsqueeze(2)).view(R, K)

        v = deq(s["a"], s["as"], M) @ deq(s["b"], s["bs"], N).t()
    else:
        def deq(q, sc, R):
            i = torch.stack((q & 15, q >> 4), 2).view(R, K // 16, 16).long()
            sig = _untiles(sc, R, K // 16).contiguous().view(torch.float8_e4m3fn).float()
            return (_e2m1_table(q.device)[i] * sig.unsqueeze(2)).view(R, K)

        ga, gb = (1.0 / ((6.0 * 448.0) / m) for m in (s["am"], s["bm"]))
        v = deq(s["a"], s["as"], M) @ deq(s["b"], s["bs"], N).t() * ga.unsqueeze(1) * gb
    if c["bias"]:
        v = v + s["bias"]
    pre = v.to(dt) if c["pre"] else None
    v = _act(v, c["act"])
    if c["residual"]:
        v = v + s["residual"].float()
    return {"out": v.to(dt), "pre": pre} if c["pre"] else {"out": v.to(dt)}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        per = (1.0 + 1.0 / 32) if case["fmt"] == 8 else (0.5 + 1.0 / 16)
        o = SIZE[case["dt"]]
        b = (M + N) * K * per + M * N * o * (1 + case["residual"] + case["pre"]) + 4 * N * case["bias"]
        return {"bytes": b, "flops": 2.0 * M * N * K}
    n, o = float(case["rows"] * case["cols"]), SIZE[case["dt"]]
    if case["op"] == "norm":
        return {"bytes": n * (o * (3 if case["residual"] else 1) + 1 + 1 / 32) + 4 * case["cols"] + 4 * case["rows"],
                "flops": 8 * n}
    if case["op"] == "norm_back":
        return {"bytes": n * o * (3 + case["dh"]) + 8 * case["cols"] + 4 * case["rows"], "flops": 11 * n}
    reads = 1 if case["act"] == "none" else 2
    return {"bytes": n * (o * (reads + case["value"]) + 2 + 2 / 32) + 4 * case["cols"] * case["bias"],
            "flops": (6 if case["act"] == "none" else 20) * n}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """run()'s values from the definitions in 64 bits (independent of the plain form)."""
    s = prepare(case, seed)
    D = torch.float64

    def two(e):
        """2^e as a double, from its bits (a library power may be off in the last one)."""
        return ((e.long() + 1023) << 52).view(D)

    def q8(v):
        """Values of the codes and of the scales of the rows of v, 32 elements a block."""
        R, C = v.shape
        b = v.reshape(R, C // 32, 32)
        m, e = torch.frexp(b.abs().amax(2) / 448.0)
        e = torch.where(m > 0.5, e, e - 1).clamp(min=-127)
        e = torch.where(m == 0, torch.full_like(e, -127), e)
        y = b * two(-e.unsqueeze(2))
        _, k = torch.frexp(y)  # |y| in [2^(k-1), 2^k): four significant bits, at least 2^-9 apart
        k = (k - 4).clamp(min=-9)
        return (torch.round(y * two(-k)) * two(k)).view(R, C), two(e)

    def tiles(v):
        """The scale values in the tiled layout, index by index; padding stands for 2^-127."""
        R, n = v.shape
        nr, nc = -(-R // 128), -(-n // 4)
        o = torch.arange(nr * nc * 512, device=v.device)
        t, j, i, k = o // 512, o % 512 // 16, o % 16 // 4, o % 4
        r, col = t // nc * 128 + 32 * i + j, t % nc * 4 + k
        ok = (r < R) & (col < n)
        return torch.where(ok, v[r.clamp(max=R - 1), col.clamp(max=n - 1)], torch.full_like(o, 2.0 ** -127, dtype=D))

    def slope(p):
        a = case["act"]
        if a == "relu":
            return torch.where(p > 0, 1.0, 0.0).to(D)
        if a == "gelu":
            return 0.5 * torch.erfc(-p / math.sqrt(2)) + p * torch.exp(-p * p / 2) / math.sqrt(2 * math.pi)
        if a == "gelu_tanh":  # p * sigma(2u)
            u2 = 2 * math.sqrt(2 / math.pi) * (p + 0.044715 * p ** 3)
            sg = torch.sigmoid(u2)
            return sg + p * sg * (1 - sg) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * p * p)
        sg = torch.sigmoid(p)
        return sg + p * sg * (1 - sg)

    if case["op"] == "norm":
        h = s["x"].to(D) + (s["residual"].to(D) if case["residual"] else 0.0)
        rstd = torch.rsqrt(torch.linalg.vector_norm(h, dim=1) ** 2 / case["cols"] + EPS)
        codes, sc = q8(h * s["weight"].to(D) * rstd[:, None])
        return {"codes": codes, "scales": tiles(sc) if case["tiled"] else sc,
                "h": h if case["residual"] else None, "rstd": rstd}
    if case["op"] == "norm_back":
        h, dy, w, r = (s[k].to(D) for k in ("h", "dy", "weight", "rstd"))
        gw = dy * w
        dx = r[:, None] * gw - (r ** 3 * (gw * h).sum(1) / case["cols"])[:, None] * h
        if case["dh"]:
            dx = dx + s["dh"].to(D)
        return {"dx": dx, "dweight": torch.mv((dy * h).t(), r)}
    if case["op"] == "quant":
        d = s["x"].to(D)
        if case["act"] != "none":
            d = d * slope(s["pre"].to(D))
        codes, sc = q8(d)
        ct, st = q8(torch.nn.functional.pad(d, (0, 0, 0, -case["rows"] % 32)).t().contiguous())
        if case["tiled"]:
            sc, st = tiles(sc), tiles(st)
        return {"codes": codes, "scales": sc, "codes_t": ct, "scales_t": st,
                "d": d if case["value"] else None, "dbias": d.sum(0) if case["bias"] else None}
    M, N, K = case["M"], case["N"], case["K"]
    blk = 32 if case["fmt"] == 8 else 16

    def values(q, tiled, R):
        nc = -(-(K // blk) // 4)
        r = torch.arange(R, device=q.device)[:, None]
        j = torch.arange(K // blk, device=q.device)[None]
        byte = tiled[((r // 128) * nc + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4]
        if blk == 32:
            sign, ex, man = q >> 7, (q >> 3 & 15).int(), (q & 7).to(D)
            v = torch.where(ex > 0, (1 + man / 8) * two(ex - 7), man / 512)
            v = torch.where(sign > 0, -v, v)
            sc = two(byte.int() - 127)
        else:
            v = torch.empty(R, K, dtype=D, device=q.device)
            t = _e2m1_table(q.device, D)
            v[:, 0::2], v[:, 1::2] = t[(q & 15).int()], t[(q >> 4).int()]
            ex, man = (byte >> 3 & 15).int(), (byte & 7).to(D)
            sc = torch.where(ex > 0, (1 + man / 8) * two(ex - 7), man / 512)
        return v * sc.repeat_interleave(blk, 1)

    v = torch.mm(values(s["a"], s["as"], M), values(s["b"], s["bs"], N).t())
    if case["fmt"] == 4:
        v = v * (s["am"].to(D) / 2688.0)[:, None] * (s["bm"].to(D) / 2688.0)
    if case["bias"]:
        v += s["bias"].to(D)
    pre = v if case["pre"] else None
    a = case["act"]
    if a == "relu":
        v = torch.where(v > 0, v, 0.0)
    elif a == "gelu":
        v = 0.5 * v * torch.erfc(-v / math.sqrt(2))
    elif a == "gelu_tanh":
        v = v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    elif a == "silu":
        v = v * torch.sigmoid(v)
    if case["residual"]:
        v = v + s["residual"].to(D)
    return {"out": v, "pre": pre} if case["pre"] else {"out": v}
