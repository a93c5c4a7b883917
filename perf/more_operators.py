"""Measured cases of the mixture-of-experts operators around the quantized products.

Tokens are packed by expert: `offs` holds the cumulative ends of the experts'
rows, rows past the last end belong to nobody and are left alone.  Four
operators, each in its plain form (elementary torch operations in 32 bits)
and, with ``own`` true, through the package's entry points:

  linear   linear8_grouped and linear4_grouped: act(a . b[e]^T + bias[e]) +
           residual, e the expert of a's row, from operands in 8 bits (32-element
           blocks) or in NVFP4 (16-element blocks); a's scales are plain, those of
           the experts' weights tiled
  quant    quantize8_grouped and act_backward_grouped: the packed rows, or the
           gradient behind an activation, in 8 bits along the rows and, each
           expert's tokens padded to 128, along the columns, with the bias
           gradients of the experts
  wgrad    linear8_grouped_wgrad: dW[e] = d[e]^T . z[e] (+ what was there) from
           the column-wise 8-bit forms
  matvec   matvec4: act(x . W[e]^T + bias[e]) + residual for few rows of 16 or 32
           bits with NVFP4 weights, one matrix or one an expert
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # up projection of one generated token with weights in 4 bits: latency
        {"name": "matvec_token", "op": "matvec", "M": 1, "X": 1, "G": 0, "used": 1, "N": 14336,
         "K": 4096, "act": "silu", "bias": True, "residual": False, "dt": "bf16"},
        # down projection of four tokens with two of eight experts each, six of them distinct
        {"name": "matvec_experts", "op": "matvec", "M": 8, "X": 8, "G": 8, "used": 6, "N": 4096,
         "K": 14336, "act": "none", "bias": False, "residual": False, "dt": "bf16"},
        # an odd batch through a narrow layer that ends inside every tile
        {"name": "matvec_odd", "op": "matvec", "M": 5, "X": 5, "G": 0, "used": 1, "N": 2064,
         "K": 1056, "act": "gelu", "bias": True, "residual": True, "dt": "f16"},
        # a decode batch over 64 experts, some of them idle: bound by the weights
        {"name": "linear4_decode", "op": "linear", "fmt": 4, "M": 256, "tail": 0, "G": 64,
         "empty": 9, "skew": 0.7, "N": 2048, "K": 7168, "act": "none", "bias": False,
         "residual": False, "pre": False, "row": False, "dt": "bf16"},
        # a prefill over the same experts, the dispatcher's buffer not full
        {"name": "linear4_prefill", "op": "linear", "fmt": 4, "M": 16384, "tail": 300, "G": 64,
         "empty": 1, "skew": 0.5, "N": 2048, "K": 7168, "act": "silu", "bias": True,
         "residual": False, "pre": False, "row": False, "dt": "bf16"},
        # up projection of a training step over eight experts, pre-activation kept
        {"name": "linear8_train", "op": "linear", "fmt": 8, "M": 8192, "tail": 0, "G": 8,
         "empty": 0, "skew": 0.3, "N": 14336, "K": 4096, "act": "gelu_tanh", "bias": True,
         "residual": False, "pre": True, "row": False, "dt": "bf16"},
        # a small ragged batch in fp16: experts that end inside every tile, one empty
        {"name": "linear8_odd", "op": "linear", "fmt": 8, "M": 1003, "tail": 17, "G": 5,
         "empty": 1, "skew": 1.0, "N": 1040, "K": 640, "act": "gelu", "bias": True,
         "residual": True, "pre": False, "row": False, "dt": "f16"},
        # the gradient behind the experts' activation, both directions, with their dbias
        {"name": "quant_act_grad", "op": "quant", "M": 8192, "tail": 0, "G": 8, "empty": 0,
         "skew": 0.3, "N": 14336, "act": "silu", "bias": True, "value": False, "dt": "bf16"},
        # the packed tokens themselves, a small fp16 batch over many experts
        {"name": "quant_tokens_odd", "op": "quant", "M": 1000, "tail": 24, "G": 16, "empty": 3,
         "skew": 1.0, "N": 2048, "act": "none", "bias": False, "value": False, "dt": "f16"},
        # the experts' weight gradients of a training step
        {"name": "wgrad_train", "op": "wgrad", "M": 8192, "tail": 0, "G": 8, "empty": 0,
         "skew": 0.3, "N": 14336, "K": 4096, "residual": False, "dt": "f32"},
        # a micro-batch added to gradients in 16 bits, idle experts keep theirs
        {"name": "wgrad_odd", "op": "wgrad", "M": 1000, "tail": 24, "G": 16, "empty": 3,
         "skew": 1.0, "N": 1056, "K": 672, "residual": True, "dt": "bf16"},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(("matvec", "linear", "linear", "quant", "wgrad"))
    dt = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "matvec":
        G = rng.choice((0, 0, 4, 8, 16, 64))
        X = _log(rng, 1, 16)
        M = X * rng.choice((1, 2, 4)) if G else X
        used = rng.randint(1, min(G, M)) if G else 1
        while True:
            N, K = _log(rng, 256, 16384, 16), _log(rng, 256, 16384, 32)
            if max(G, 1) * N * K <= 8 * 4096 * 14336 and used * N * K <= 6 * 4096 * 14336:
                break
        return {"op": op, "M": M, "X": X, "G": G, "used": used, "N": N, "K": K,
                "act": rng.choice(ACTS), "bias": rng.random() < 0.5,
                "residual": rng.random() < 0.4, "dt": dt}
    M = _log(rng, 1, 16384)
    tail = rng.choice((0, 0, min(M - 1, rng.randint(0, 200))))
    G = _log(rng, 1, 64)
    empty = rng.choice((0, rng.randint(0, G - 1)))
    empty = max(empty, G - (M - tail))
    c = {"op": op, "M": M, "tail": tail, "G": G, "empty": empty, "skew": rng.choice((0.0, 0.5, 1.0))}
    if op == "quant":
        N = _log(rng, 256, 16384, 32)
        while M * N > 8192 * 14336:
            N = N // 64 * 32
        act = rng.choice(ACTS)
        if dt == "f32" and M * N > 8192 * 7168:
            dt = "bf16"
        c.update(N=N, act=act, bias=act != "none" and rng.random() < 0.7,
                 value=act != "none" and rng.random() < 0.3, dt=dt)
        return c
    fmt = rng.choice((8, 4)) if op == "linear" else 8
    while True:
        if op == "linear":
            N, K = _log(rng, 256, 16384, 16), _log(rng, 256, 16384, 128 if fmt == 8 else 64)
        else:
            N, K = _log(rng, 256, 16384, 32), _log(rng, 256, 16384, 32)
        if G * N * K <= 8 * 14336 * 4096 and M * N * K <= 8192 * 14336 * 4096 and M * N <= 8192 * 14336:
            break
    c.update(N=N, K=K, residual=rng.random() < 0.5, dt=dt)
    if op == "linear":
        c.update(fmt=fmt, act=rng.choice(ACTS), bias=rng.random() < 0.5, pre=rng.random() < 0.3,
                 row=fmt == 4 and rng.random() < 0.4)
    return c


# ------------------------------------------------------------------ shared plain pieces
def _ends(case, seed):
    """Cumulative ends of the experts' rows: `empty` of the G experts have none,
    the others at least one, sizes log-normally spread."""
    rng = random.Random(seed * 7919 + 17)
    G, total = case["G"], case["M"] - case["tail"]
    idle = set(rng.sample(range(G), case["empty"]))
    busy = [g for g in range(G) if g not in idle]
    w = [math.exp(case["skew"] * rng.gauss(0, 1)) for _ in busy]
    spare, sizes = total - len(busy), {}
    cum, s = 0.0, 0
    for g, x in zip(busy, w):
        cum += x
        upto = int(round(spare * cum / sum(w)))
        sizes[g] = 1 + upto - s
        s = upto
    ends, e = [], 0
    for g in range(G):
        e += sizes.get(g, 0)
        ends.append(e)
    return ends


def _pad_cols(rows, G):
    """Columns of a column-wise form: every expert's rows padded to a multiple of 128."""
    return (rows + 127 * min(G, rows)) // 128 * 128


def _spans(ends):
    """(expert, first row, end row, first padded column, padded end)."""
    out, r, p = [], 0, 0
    for g, e in enumerate(ends):
        q = p + (e - r + 127) // 128 * 128
        out.append((g, r, e, p, q))
        r, p = e, q
    return out


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


def _from8(codes, scales):
    """fp32 values of E4M3 codes [R, C] (bytes) and plain scales [R, C/32]."""
    R, C = codes.shape
    two = (scales.int() << 23).view(torch.float32)
    return (codes.view(torch.float8_e4m3fn).float().view(R, C // 32, 32) * two.unsqueeze(2)).view(R, C)


def _from4(codes, scales):
    """fp32 values (without the global scale) of E2M1 codes and plain E4M3 scales."""
    R, C = codes.shape[0], codes.shape[1] * 2
    i = torch.stack((codes & 15, codes >> 4), 2).view(R, C // 16, 16).long()
    sig = scales.contiguous().view(torch.float8_e4m3fn).float()
    return (_e2m1_table(codes.device)[i] * sig.unsqueeze(2)).view(R, C)


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


def _nvfp4(x, amax):
    """Standard NVFP4 operand of fp32 x under amax ([rows] or [1]): codes, plain scale bytes."""
    R, C = x.shape
    Sr = ((6.0 * 448.0) / amax).view(-1, 1, 1)
    b = x.view(R, C // 16, 16)
    s8 = ((b.abs().amax(2, keepdim=True) * Sr) / 6.0).to(torch.float8_e4m3fn)
    sig = s8.float()
    y = torch.where(sig > 0, b * (Sr / sig), torch.zeros_like(b))
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    mag = torch.bucketize(y.abs(), edges).to(torch.uint8)
    code = (mag | (torch.signbit(y).to(torch.uint8) << 3)).view(R, C // 2, 2)
    return (code[:, :, 0] | (code[:, :, 1] << 4)).contiguous(), s8.view(torch.uint8).view(R, C // 16)


# ------------------------------------------------------------------ inputs
def _acts(g, rows, cols):
    """Activation-like values: N(0, 1) with one entry in a thousand 20 times as large."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    return torch.where(torch.rand(rows, cols, generator=g, device=DEV) < 1e-3, x * 20.0, x)


def _weights4(g, G, N, K):
    """NVFP4 weights of G experts: codes [G, N, K/2], tiled scales [G, bytes], amax [G]."""
    codes, scales, amax = [], [], []
    for _ in range(G):
        w = torch.randn(N, K, generator=g, device=DEV) * 0.02
        m = w.abs().amax().view(1)
        c, s = _nvfp4(w, m)
        codes.append(c)
        scales.append(_tiles(s))
        amax.append(m)
    return torch.stack(codes), torch.stack(scales), torch.cat(amax)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    dt, op, M, N = DT[case["dt"]], case["op"], case["M"], case["N"]
    s = {"case": case}
    if op == "matvec":
        K, G, X = case["K"], case["G"], case["X"]
        s["x"] = _acts(g, X, K).to(dt)
        s["b"], s["bs"], s["bm"] = _weights4(g, max(G, 1), N, K)
        if G:
            rng = random.Random(int(seed) + 5)
            some = rng.sample(range(G), case["used"])
            ids = some + [rng.choice(some) for _ in range(M - len(some))]
            rng.shuffle(ids)
            s["ids_list"] = ids
            s["ids"] = torch.tensor(ids, dtype=torch.int32, device=DEV)
        else:
            s["b"], s["bs"], s["ids"] = s["b"][0], s["bs"][0], None
        n = max(G, 1)
        s["bias"] = (torch.randn(n, N, generator=g, device=DEV) * 0.5) if case["bias"] else None
        if case["bias"] and not G:
            s["bias"] = s["bias"][0]
        s["residual"] = torch.randn(M, N, generator=g, device=DEV).to(dt) if case["residual"] else None
        s["out"] = torch.empty(M, N, dtype=dt, device=DEV)
        return s
    G, ends = case["G"], _ends(case, int(seed))
    s["ends"] = ends
    s["offs"] = torch.tensor(ends, dtype=torch.int32, device=DEV)
    if op == "linear":
        K = case["K"]
        a = _acts(g, M, K)
        if case["fmt"] == 8:
            c, s["as"] = _mx8(a)
            s["a"] = c.view(torch.uint8)
            codes, scales = [], []
            for _ in range(G):
                c, sc = _mx8(torch.randn(N, K, generator=g, device=DEV) * 0.02)
                codes.append(c.view(torch.uint8))
                scales.append(_tiles(sc))
            s["b"], s["bs"] = torch.stack(codes), torch.stack(scales)
        else:
            row = a.abs().amax(1)
            if case["row"]:
                s["am"] = per = row
            else:
                per, s["am"] = row.clone(), torch.ones(G, device=DEV)
                for e, r0, r1, _, _ in _spans(ends):
                    if r1 > r0:
                        s["am"][e] = row[r0:r1].amax()
                        per[r0:r1] = s["am"][e]
            s["a"], s["as"] = _nvfp4(a, per)
            s["b"], s["bs"], s["bm"] = _weights4(g, G, N, K)
        s["bias"] = (torch.randn(G, N, generator=g, device=DEV) * 0.5) if case["bias"] else None
        s["residual"] = torch.randn(M, N, generator=g, device=DEV).to(dt) if case["residual"] else None
        s["out"] = torch.zeros(M, N, dtype=dt, device=DEV)
        s["pre"] = torch.zeros(M, N, dtype=dt, device=DEV) if case["pre"] else None
        return s
    P = _pad_cols(M, G)
    if op == "quant":
        if case["act"] == "none":
            s["x"] = _acts(g, M, N).to(dt)
        else:
            s["x"] = (torch.randn(M, N, generator=g, device=DEV) * 0.05).to(dt)
            s["pre"] = (torch.randn(M, N, generator=g, device=DEV) * 1.5).to(dt)
        z8 = lambda *n: torch.zeros(*n, dtype=torch.uint8, device=DEV)  # noqa: E731
        s["codes"], s["scales"] = z8(M, N), z8(M, N // 32)
        s["codes_t"], s["scales_t"] = z8(N, P), z8((N + 127) // 128 * P // 128 * 512)
        s["d"] = torch.zeros(M, N, dtype=dt, device=DEV) if case["value"] else None
        s["dbias"] = torch.empty(G, N, device=DEV) if case["bias"] else None
        return s
    K = case["K"]
    for name, n, scale in (("d", N, 0.05), ("z", K, 1.0)):
        t = torch.zeros(n, P, device=DEV)
        for _, r0, r1, p0, _ in _spans(ends):
            if r1 > r0:
                t[:, p0:p0 + r1 - r0] = torch.randn(n, r1 - r0, generator=g, device=DEV) * scale
        c, sc = _mx8(t)
        s[name], s[name + "s"] = c.view(torch.uint8), _tiles(sc)
    s["residual"] = (torch.randn(G, N, K, generator=g, device=DEV) * 2).to(dt) if case["residual"] else None
    s["out"] = torch.empty(G, N, K, dtype=dt, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import nvfp4_quantization_precision_gb300 as fos
    c = s["case"]
    dt = DT[c["dt"]]
    if c["op"] == "matvec":
        return {"out": fos.matvec4(s["x"], s["b"], s["bs"], s["bm"], ids=s["ids"], act=c["act"],
                                   bias=s["bias"], residual=s["residual"], out_dtype=dt,
                                   out=s["out"])}
    if c["op"] == "linear":
        more = {"act": c["act"], "bias": s["bias"], "residual": s["residual"], "out_dtype": dt,
                "save_pre": c["pre"], "out": s["out"], "pre": s["pre"]}
        if c["fmt"] == 8:
            r = fos.linear8_grouped(s["a"], s["as"], s["b"], s["bs"], s["offs"], **more)
        else:
            r = fos.linear4_grouped(s["a"], s["as"], s["am"], s["b"], s["bs"], s["bm"], s["offs"],
                                    cfg=fos.Config(row_scaled=c["row"]), **more)
        return {"out": r[0], "pre": r[1]} if c["pre"] else {"out": r}
    if c["op"] == "quant":
        buf = {k: s[k] for k in ("codes", "scales", "codes_t", "scales_t")}
        if c["act"] == "none":
            q = fos.quantize8_grouped(s["x"], s["offs"], **buf)
            d = dbias = None
        else:
            *q, d, dbias = fos.act_backward_grouped(
                s["x"], s["pre"], c["act"], s["offs"], value=c["value"], bias_grad=c["bias"],
                d=s["d"], dbias=s["dbias"], **buf)
        codes, scales = _held(q[0], q[1])
        codes_t, scales_t = _held(q[2], q[3])
        return {"codes": codes, "scales": scales, "codes_t": codes_t, "scales_t": scales_t,
                "d": d, "dbias": dbias}
    return {"out": fos.linear8_grouped_wgrad(s["d"], s["ds"], s["z"], s["zs"], s["offs"], c["M"],
                                             residual=s["residual"], out_dtype=dt, out=s["out"])}


def _run_plain(s):
    c = s["case"]
    dt, op, M, N = DT[c["dt"]], c["op"], c["M"], c["N"]
    if op == "matvec":
        K, G, per = c["K"], c["G"], c["M"] // c["X"]
        x = s["x"].float().repeat_interleave(per, 0)
        gb = 1.0 / ((6.0 * 448.0) / s["bm"])
        v = torch.zeros(M, N, device=x.device)
        if not G:
            v = x @ _from4(s["b"], _untiles(s["bs"], N, K // 16)).t() * gb
            if c["bias"]:
                v = v + s["bias"]
        else:
            for e in sorted(set(s["ids_list"])):
                at = (s["ids"] == e).unsqueeze(1)
                y = x @ _from4(s["b"][e], _untiles(s["bs"][e], N, K // 16)).t() * gb[e]
                v = torch.where(at, y + s["bias"][e] if c["bias"] else y, v)
        v = _act(v, c["act"])
        if c["residual"]:
            v = v + s["residual"].float()
        return {"out": v.to(dt)}
    spans = _spans(s["ends"])
    if op == "linear":
        K = c["K"]
        out = torch.zeros(M, N, dtype=dt, device=s["a"].device)
        pre = torch.zeros_like(out) if c["pre"] else None
        if c["fmt"] == 4:
            ga, gb = (1.0 / ((6.0 * 448.0) / m) for m in (s["am"], s["bm"]))
        for e, r0, r1, _, _ in spans:
            if r1 == r0:
                continue
            if c["fmt"] == 8:
                v = _from8(s["a"][r0:r1], s["as"][r0:r1]) @ _from8(s["b"][e], _untiles(s["bs"][e], N, K // 32)).t()
            else:
                v = (_from4(s["a"][r0:r1], s["as"][r0:r1])
                     @ _from4(s["b"][e], _untiles(s["bs"][e], N, K // 16)).t())
                v = v * (ga[r0:r1].unsqueeze(1) if c["row"] else ga[e]) * gb[e]
            if c["bias"]:
                v = v + s["bias"][e]
            if c["pre"]:
                pre[r0:r1] = v.to(dt)
            v = _act(v, c["act"])
            if c["residual"]:
                v = v + s["residual"][r0:r1].float()
            out[r0:r1] = v.to(dt)
        return {"out": out, "pre": pre} if c["pre"] else {"out": out}
    if op == "quant":
        d = s["x"].float()
        if c["act"] != "none":
            d = d * _act_slope(s["pre"].float(), c["act"])
        end = s["ends"][-1]
        codes, sc = torch.zeros_like(s["codes"]), torch.zeros_like(s["scales"])
        q, qs = _mx8(d[:end])
        codes[:end], sc[:end] = q.view(torch.uint8), qs
        t = torch.zeros(N, s["codes_t"].shape[1], device=d.device)
        dbias = torch.zeros(c["G"], N, device=d.device) if c["bias"] else None
        for e, r0, r1, p0, _ in spans:
            if r1 > r0:
                t[:, p0:p0 + r1 - r0] = d[r0:r1].t()
                if c["bias"]:
                    dbias[e] = d[r0:r1].sum(0)
        codes_t, sct = _mx8(t)
        dv = None
        if c["value"]:
            dv = torch.zeros_like(s["x"])
            dv[:end] = d[:end].to(dt)
        codes, scales = _held(codes, sc)
        codes_t, scales_t = _held(codes_t, _tiles(sct))
        return {"codes": codes, "scales": scales, "codes_t": codes_t, "scales_t": scales_t,
                "d": dv, "dbias": dbias}
    K, P = c["K"], s["d"].shape[1]
    d, z = _from8(s["d"], _untiles(s["ds"], N, P // 32)), _from8(s["z"], _untiles(s["zs"], K, P // 32))
    out = torch.zeros(c["G"], N, K, dtype=dt, device=d.device)
    for e, r0, r1, p0, p1 in spans:
        v = d[:, p0:p1] @ z[:, p0:p1].t()
        if c["residual"]:
            v = v + s["residual"][e].float()
        out[e] = v.to(dt)
    return {"out": out}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, M, N, o = case["op"], case["M"], case["N"], SIZE[case["dt"]]
    if op == "matvec":
        K = case["K"]
        return {"bytes": case["used"] * (N * K * 0.5625 + 4 * N * case["bias"]) + case["X"] * K * o
                + M * N * o * (1 + case["residual"]), "flops": 2.0 * M * N * K}
    T, busy = M - case["tail"], case["G"] - case["empty"]
    if op == "linear":
        K = case["K"]
        per = (1.0 + 1.0 / 32) if case["fmt"] == 8 else (0.5 + 1.0 / 16)
        return {"bytes": (T + busy * N) * K * per + T * N * o * (1 + case["residual"] + case["pre"])
                + 4 * busy * N * case["bias"], "flops": 2.0 * T * N * K}
    if op == "quant":
        reads = 1 if case["act"] == "none" else 2
        n = float(T * N)
        return {"bytes": n * (o * (reads + case["value"]) + 2 + 2 / 32) + 4 * case["G"] * N * case["bias"],
                "flops": (6 if case["act"] == "none" else 20) * n}
    K, G = case["K"], case["G"]
    return {"bytes": (N + K) * T * (1 + 1 / 32) + G * N * K * o * (1 + case["residual"]),
            "flops": 2.0 * T * N * K}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """run()'s values from the definitions in 64 bits (independent of the plain form)."""
    s = prepare(case, seed)
    D = torch.float64
    op, M, N = case["op"], case["M"], case["N"]

    def two(e):
        """2^e as a double, from its bits (a library power may be off in the last one)."""
        return ((e.long() + 1023) << 52).view(D)

    def e4m3(q):
        sign, ex, man = q >> 7, (q >> 3 & 15).int(), (q & 7).to(D)
        v = torch.where(ex > 0, (1 + man / 8) * two(ex - 7), man / 512)
        return torch.where(sign > 0, -v, v)

    def tiled_bytes(tiled, R, n):
        nc = -(-n // 4)
        r = torch.arange(R, device=tiled.device)[:, None]
        j = torch.arange(n, device=tiled.device)[None]
        return tiled[((r // 128) * nc + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4]

    def values8(q, byte):
        return e4m3(q) * two(byte.int() - 127).repeat_interleave(32, 1)

    def values4(q, byte):
        v = torch.empty(q.shape[0], q.shape[1] * 2, dtype=D, device=q.device)
        t = _e2m1_table(q.device, D)
        v[:, 0::2], v[:, 1::2] = t[(q & 15).int()], t[(q >> 4).int()]
        return v * e4m3(byte).repeat_interleave(16, 1)

    def act(v):
        a = case["act"]
        if a == "relu":
            return torch.where(v > 0, v, 0.0)
        if a == "gelu":
            return 0.5 * v * torch.erfc(-v / math.sqrt(2))
        if a == "gelu_tanh":
            return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
        return v * torch.sigmoid(v) if a == "silu" else v

    def slope(p):
        a = case["act"]
        if a == "relu":
            return torch.where(p > 0, 1.0, 0.0).to(D)
        if a == "gelu":
            return 0.5 * torch.erfc(-p / math.sqrt(2)) + p * torch.exp(-p * p / 2) / math.sqrt(2 * math.pi)
        if a == "gelu_tanh":
            u2 = 2 * math.sqrt(2 / math.pi) * (p + 0.044715 * p ** 3)
            sg = torch.sigmoid(u2)
            return sg + p * sg * (1 - sg) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * p * p)
        sg = torch.sigmoid(p)
        return sg + p * sg * (1 - sg)

    if op == "matvec":
        K, per = case["K"], M // case["X"]
        v = torch.zeros(M, N, dtype=D, device=DEV)
        ids = s["ids_list"] if case["G"] else [0] * M
        for e in set(ids):
            b, bs = (s["b"][e], s["bs"][e]) if case["G"] else (s["b"], s["bs"])
            w = values4(b, tiled_bytes(bs, N, K // 16)) * (s["bm"][e].to(D) / 2688.0)
            rows = [p for p in range(M) if ids[p] == e]
            v[rows] = torch.mm(s["x"][[p // per for p in rows]].to(D), w.t())
            if case["bias"]:
                v[rows] += (s["bias"][e] if case["G"] else s["bias"]).to(D)
        v = act(v)
        if case["residual"]:
            v = v + s["residual"].to(D)
        return {"out": v}
    lo = [0] + s["ends"][:-1]
    if op == "linear":
        K, fmt = case["K"], case["fmt"]
        out = torch.zeros(M, N, dtype=D, device=DEV)
        pre = torch.zeros_like(out) if case["pre"] else None
        for e, (r0, r1) in enumerate(zip(lo, s["ends"])):
            if r0 == r1:
                continue
            if fmt == 8:
                v = torch.mm(values8(s["a"][r0:r1], s["as"][r0:r1]),
                             values8(s["b"][e], tiled_bytes(s["bs"][e], N, K // 32)).t())
            else:
                v = torch.mm(values4(s["a"][r0:r1], s["as"][r0:r1]),
                             values4(s["b"][e], tiled_bytes(s["bs"][e], N, K // 16)).t())
                am = s["am"][r0:r1, None] if case["row"] else s["am"][e]
                v *= (am.to(D) / 2688.0) * (s["bm"][e].to(D) / 2688.0)
            if case["bias"]:
                v += s["bias"][e].to(D)
            if case["pre"]:
                pre[r0:r1] = v
            v = act(v)
            if case["residual"]:
                v = v + s["residual"][r0:r1].to(D)
            out[r0:r1] = v
        return {"out": out, "pre": pre} if case["pre"] else {"out": out}
    # first padded column of each expert
    at, p = [], 0
    for r0, r1 in zip(lo, s["ends"]):
        at.append(p)
        p += -(-(r1 - r0) // 128) * 128
    if op == "quant":
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
            return torch.where(ok, v[r.clamp(max=R - 1), col.clamp(max=n - 1)],
                               torch.full_like(o, 2.0 ** -127, dtype=D))

        d = s["x"].to(D)
        if case["act"] != "none":
            d = d * slope(s["pre"].to(D))
        d[s["ends"][-1]:] = 0.0  # nobody's rows: the buffers' zeros
        codes, sc = q8(d)
        cols = torch.zeros(s["codes_t"].shape[1], N, dtype=D, device=DEV)
        dbias = torch.zeros(case["G"], N, dtype=D, device=DEV) if case["bias"] else None
        for e, (r0, r1) in enumerate(zip(lo, s["ends"])):
            cols[at[e]:at[e] + r1 - r0] = d[r0:r1]
            if case["bias"]:
                dbias[e] = d[r0:r1].sum(0)
        ct, st = q8(cols.t().contiguous())
        return {"codes": codes, "scales": sc, "codes_t": ct, "scales_t": tiles(st),
                "d": d if case["value"] else None, "dbias": dbias}
    K, P = case["K"], s["d"].shape[1]
    d = values8(s["d"], tiled_bytes(s["ds"], N, P // 32))
    z = values8(s["z"], tiled_bytes(s["zs"], K, P // 32))
    out = torch.empty(case["G"], N, K, dtype=D, device=DEV)
    for e, (r0, r1) in enumerate(zip(lo, s["ends"])):
        k = slice(at[e], at[e] + r1 - r0)
        torch.mm(d[:, k], z[:, k].t(), out=out[e])
        if case["residual"]:
            out[e] += s["residual"][e].to(D)
    return {"out": out}
