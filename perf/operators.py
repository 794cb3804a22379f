"""Operators around the library's block-scaled linear layers, as timed and compared cases.

Six operators in one set: what makes a block-scaled product's operand (``norm``, ``quant``), what a training step
does with the 8-bit operand that it kept (``wgrad``, and the norm's backward ``bwd``), and the product of a few
tokens with 4-bit weights (``gemv``).  With ``own`` false each runs in its plain form, elementary torch operations
in 32 bits; with ``own`` true through the package's entry points.

Definitions (e4m3 codes q with one power-of-two scale 2^e per 32 consecutive elements of a row):
  quantise  e = the least integer with max|x| <= 448 * 2^e in the block (at least -127); q = x / 2^e rounded to
            nearest even
  norm      h = x + r rounded to x's type; rstd = 1 / sqrt(mean(h^2) + eps); y = h * rstd * w, given out in x's
            type or quantised
  bwd       g = dy * w;  dx = dh + rstd * g - h * rstd^3 * mean(g * h);  dw = sum over rows of dy * h * rstd
  wgrad     dw[m, n] = c[m, n] + sum over tokens t of dy[t, m] * q[t, n] * 2^e[t, n / 32]
  gemv      d[m, n] = sum over k of x[m, k] * e2m1[n, k] * 2^s[n, k / kblock]
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "f32": 4}


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one token of a decode step: the norm between two layers, whose row the products with 4-bit weights read
        dict(name="norm_token_bf16", op="norm", rows=1, n=4096, type="bf16", residual=True, out="same"),
        # a prompt or training batch: the norm in front of a block-scaled projection, its operand made on the way
        dict(name="norm_prompt_mxfp8", op="norm", rows=16384, n=4096, type="bf16", residual=True, out="mxfp8"),
        # the same batch's backward pass, with the gradient that arrives on the residual stream
        dict(name="bwd_batch_bf16", op="bwd", rows=16384, n=4096, type="bf16", dh=True),
        # a ragged batch with an fp32 residual stream
        dict(name="bwd_ragged_f32", op="bwd", rows=1001, n=4100, type="f32", dh=False),
        # the wide activation of a feed-forward block, kept in 8 bits
        dict(name="quant_wide_bf16", op="quant", rows=16384, n=14336, type="bf16"),
        # a short sequence's activation
        dict(name="quant_short_fp16", op="quant", rows=333, n=4096, type="fp16"),
        # weight gradient of a feed-forward projection over a full batch
        dict(name="wgrad_wide", op="wgrad", m=14336, n=4096, k=16384, out="f32", acc=False),
        # square projection, ragged token count, added to the gradient of earlier micro-batches
        dict(name="wgrad_ragged_acc", op="wgrad", m=4096, n=4096, k=4100, out="f32", acc=True),
        # a narrow projection: few output tiles, long sum over tokens
        dict(name="wgrad_narrow", op="wgrad", m=1024, n=992, k=8200, out="bf16", acc=False),
        # one token through a feed-forward projection
        dict(name="gemv_token_bf16", op="gemv", m=1, n=14336, k=4096, kblock=32, type="bf16", out="bf16"),
        # a batch of 16 sequences, one token each, the projection back; wider groups, fp32 result
        dict(name="gemv_batch16_fp16", op="gemv", m=16, n=4096, k=14336, kblock=128, type="fp16", out="f32"),
        # the output projection onto a vocabulary, four sequences
        dict(name="gemv_vocab_bf16", op="gemv", m=4, n=131072, k=8192, kblock=32, type="bf16", out="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "bwd", "quant", "wgrad", "gemv"])
    if op == "norm":
        out = rng.choice(["same", "mxfp8"])
        n = 32 * _log(rng, 2, 512) if out == "mxfp8" else _log(rng, 64, 16384)
        return dict(op=op, rows=_log(rng, 1, 16384), n=n, type=rng.choice(list(TYPES)),
                    residual=rng.random() < 0.7, out=out)
    if op == "bwd":
        return dict(op=op, rows=_log(rng, 1, 16384), n=_log(rng, 64, 16384), type=rng.choice(list(TYPES)),
                    dh=rng.random() < 0.7)
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 16384), n=32 * _log(rng, 1, 448), type=rng.choice(list(TYPES)))
    if op == "wgrad":
        m = 8 * _log(rng, 2, 1792) if rng.random() < 0.8 else _log(rng, 16, 4096)
        return dict(op=op, m=m, n=32 * _log(rng, 1, 128), k=_log(rng, 1, 16384), out=rng.choice(["f32", "bf16"]),
                    acc=rng.random() < 0.4)
    k = 32 * _log(rng, 2, 512)
    return dict(op=op, m=_log(rng, 1, 32), n=_log(rng, 16, 65536), k=k, kblock=rng.choice([32, 64, 128, k]),
                type=rng.choice(["bf16", "fp16"]), out=rng.choice(["f32", "bf16"]))


# ---- inputs -----------------------------------------------------------------

def _activations(g, rows, n, dtype):
    """A hidden state: unit noise with a few columns many times larger, as trained models show them."""
    x = torch.randn(rows, n, generator=g, device=g.device)
    big = torch.rand(n, generator=g, device=g.device) < 0.005
    return torch.where(big, x * 20, x).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda" if torch.cuda.is_available() else "cpu")
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    dev, op = g.device, case["op"]
    s = dict(case)

    def noise(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def room(*shape, dtype):
        return torch.empty(*shape, dtype=dtype, device=dev)

    if op == "norm":
        t = TYPES[case["type"]]
        rows, n = case["rows"], case["n"]
        s["x"] = _activations(g, rows, n, t)
        s["r"] = _activations(g, rows, n, t) if case["residual"] else None
        s["w"] = (1 + 0.1 * noise(n)).to(t)
        s["h"] = room(rows, n, dtype=t) if case["residual"] else None
        s["rstd"] = room(rows, dtype=torch.float32)
        if case["out"] == "mxfp8":
            s["q"], s["sf"] = room(rows, n, dtype=torch.float8_e4m3fn), room(rows, n // 32, dtype=torch.float8_e8m0fnu)
        else:
            s["y"] = room(rows, n, dtype=t)
    elif op == "bwd":
        t = TYPES[case["type"]]
        rows, n = case["rows"], case["n"]
        s["h"] = _activations(g, rows, n, t)
        s["w"] = (1 + 0.1 * noise(n)).to(t)
        s["dy"] = (0.01 * noise(rows, n)).to(t)
        s["dh"] = (0.01 * noise(rows, n)).to(t) if case["dh"] else None
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
        s["dx"], s["dw"] = room(rows, n, dtype=t), room(n, dtype=torch.float32)
        s["ws"] = room(64 << 20, dtype=torch.uint8)      # room for partial sums, kept for the program's life
    elif op == "quant":
        rows, n = case["rows"], case["n"]
        # what a gated feed-forward block hands on: a product of two, with a heavy tail
        s["x"] = (torch.nn.functional.silu(noise(rows, n)) * noise(rows, n)).to(TYPES[case["type"]])
        s["q"], s["sf"] = room(rows, n, dtype=torch.float8_e4m3fn), room(rows, n // 32, dtype=torch.float8_e8m0fnu)
    elif op == "wgrad":
        m, n, k = case["m"], case["n"], case["k"]
        t = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        s["dy"] = (0.01 * noise(k, m)).to(torch.bfloat16)
        s["q"], s["sf"] = _quantize(noise(k, n))
        s["c"] = noise(m, n).to(t) if case["acc"] else None
        s["d"] = room(m, n, dtype=t)
        s["ws"] = room(256 << 20, dtype=torch.uint8)
    else:
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = noise(m, k).to(TYPES[case["type"]])
        s["w"] = torch.randint(0, 256, (n, k // 2), generator=g, device=dev, dtype=torch.uint8)
        s["sf"] = torch.randint(116, 122, (n, -(-k // case["kblock"])), generator=g, device=dev, dtype=torch.uint8)
        s["d"] = room(m, n, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    return s


# ---- plain forms and calls --------------------------------------------------

def _quantize(x):
    """(codes as float8_e4m3fn, scales as float8_e8m0fnu) of the rows of fp32 x."""
    rows, n = x.shape
    b = x.reshape(rows, n // 32, 32)
    frac, power = torch.frexp(b.abs().amax(2))           # amax = frac * 2^power, 0.5 <= frac < 1
    e = (power - 9 + (frac > 0.875).int()).clamp_min(-127)
    q = torch.ldexp(b, -e.unsqueeze(2)).to(torch.float8_e4m3fn).reshape(rows, n)
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _norm(s):
    x, w = s["x"], s["w"].float()
    h = x if s["r"] is None else (x.float() + s["r"].float()).to(x.dtype)
    f = h.float()
    rstd = torch.rsqrt(f.square().mean(1) + EPS)
    y = f * w * rstd[:, None]
    if s["out"] == "mxfp8":
        return (*_quantize(y), h, rstd)
    return y.to(x.dtype), h, rstd


def _bwd(s):
    dy, h, rstd = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
    g = dy * s["w"].float()
    dx = rstd * g - h * (rstd * rstd * rstd * (g * h).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dx.to(s["dy"].dtype), (dy * h * rstd).sum(0)


def _wgrad(s):
    k, n = s["q"].shape
    x = (s["q"].float().reshape(k, n // 32, 32) * s["sf"].float()[:, :, None]).reshape(k, n)
    d = torch.mm(s["dy"].float().t(), x)
    if s["c"] is not None:
        d = d + s["c"].float()
    return d.to(s["d"].dtype)


# the two e2m1 values of each byte, low nibble first
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
_PAIRS = [[_E2M1[b & 15], _E2M1[b >> 4]] for b in range(256)]


def _gemv(s):
    n, k, kb = s["n"], s["k"], s["kblock"]
    w = torch.tensor(_PAIRS, device=s["w"].device)[s["w"].int()].reshape(n, k)
    scale = torch.ldexp(torch.ones((), device=w.device), s["sf"].int() - 127)
    if k % kb == 0:
        w = (w.reshape(n, k // kb, kb) * scale[:, :, None]).reshape(n, k)
    else:
        w = w * scale.repeat_interleave(kb, 1)[:, :k]
    return torch.mm(s["x"].float(), w.t()).to(s["d"].dtype)


def run(state):
    s, op = state, state["op"]
    if not own:
        return {"norm": _norm, "bwd": _bwd, "wgrad": _wgrad, "gemv": _gemv,
                "quant": lambda s: _quantize(s["x"].float())}[op](s)
    import tiled_dense_gemm_tile_amd as tg
    if op == "norm":
        if s["out"] == "mxfp8":
            return tg.rmsnorm_mxfp8(s["x"], s["w"], EPS, residual=s["r"], Q=s["q"], SF=s["sf"], H=s["h"],
                                    rstd=s["rstd"])
        return tg.rmsnorm(s["x"], s["w"], EPS, residual=s["r"], Y=s["y"], H=s["h"], rstd=s["rstd"])
    if op == "bwd":
        return tg.rmsnorm_backward(s["dy"], s["h"], s["w"], s["rstd"], dH=s["dh"], dX=s["dx"], dW=s["dw"],
                                   workspace=s["ws"])
    if op == "quant":
        return tg.mxfp8_quantize(s["x"], Q=s["q"], SF=s["sf"])
    if op == "wgrad":
        return tg.gemm_wgrad_mxfp8(s["dy"], s["q"], s["sf"], C=s["c"], D=s["d"], out_dtype=s["d"].dtype,
                                   workspace=s["ws"])
    return tg.gemv_mxfp4(s["x"], s["w"], s["sf"], kblock=s["kblock"], D=s["d"], out_dtype=s["d"].dtype)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    op = case["op"]
    if op == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * k // 2 + n * -(-k // case["kblock"]) + m * k * 2 + m * n * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * m * n * k}
    if op == "wgrad":
        m, n, k = case["m"], case["n"], case["k"]
        o = 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * k * m + k * n + k * (n // 32) + m * n * o * (2 if case["acc"] else 1), "flops": 2 * m * n * k}
    rows, n = case["rows"], case["n"]
    e, z = rows * n, SIZE[case["type"]]
    if op == "quant":
        return {"bytes": e * z + e + e // 32, "flops": 3 * e}
    if op == "bwd":
        return {"bytes": e * z * (4 if case["dh"] else 3) + n * z + 4 * n + 4 * rows, "flops": 10 * e}
    out = e + e // 32 if case["out"] == "mxfp8" else e * z
    return {"bytes": e * z * (3 if case["residual"] else 1) + out + n * z + 4 * rows, "flops": 6 * e}


# ---- the definitions in 64 bits ---------------------------------------------

def _nearest(v, bits, low):
    """float64 v rounded to nearest even at `bits` bits after the leading one, no finer than 2^(low - bits)."""
    p = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** (low - 60))))
    p = torch.where(torch.exp2(p + 1) <= v.abs(), p + 1, torch.where(torch.exp2(p) > v.abs(), p - 1, p))
    step = torch.exp2(p.clamp_min(low) - bits)
    return torch.round(v / step) * step


def _blocks(v):
    """(code values, scales) in float64 of the rows of float64 v."""
    rows, n = v.shape
    b = v.reshape(rows * (n // 32), 32)
    top = b.abs().max(1).values
    e = torch.floor(torch.log2((top / 448).clamp_min(2.0 ** -127)))
    e = torch.where(448 * torch.exp2(e) < top, e + 1, e)
    scale = torch.exp2(e)
    return _nearest(b / scale[:, None], 3, -6).reshape(rows, n), scale.reshape(rows, n // 32)


_FORMAT = {"bf16": (7, -126), "fp16": (10, -14), "f32": (23, -126)}


def _e4m3_value(codes):
    c = codes.view(torch.uint8).to(torch.int16)
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2(e.double() - 10))
    return torch.where(c >= 128, -v, v)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quant":
        return _blocks(s["x"].double())
    if op == "norm":
        h = s["x"].double()
        if s["r"] is not None:
            h = _nearest(h + s["r"].double(), *_FORMAT[case["type"]])
        rstd = 1 / torch.sqrt(torch.sum(h * h, 1) / case["n"] + EPS)
        y = h * (rstd[:, None] * s["w"].double())
        return (*_blocks(y), h, rstd) if case["out"] == "mxfp8" else (y, h, rstd)
    if op == "bwd":
        dy, h, w = s["dy"].double(), s["h"].double(), s["w"].double()
        unit = h * s["rstd"].double()[:, None]           # the normed row, before its weight
        through = torch.sum(dy * w * unit, 1, keepdim=True) / case["n"]
        dx = (dy * w - unit * through) * s["rstd"].double()[:, None]
        return dx + (0 if s["dh"] is None else s["dh"].double()), torch.sum(dy * unit, 0)
    if op == "wgrad":
        scale = torch.exp2(s["sf"].view(torch.uint8).double() - 127)
        x = _e4m3_value(s["q"]) * torch.repeat_interleave(scale, 32, 1)
        d = s["dy"].double().t().contiguous() @ x
        return d if s["c"] is None else d + s["c"].double()
    x, n, k = s["x"].double(), case["n"], case["k"]
    parts = []
    for lo in range(0, n, 16384):                        # a slab of weight rows at a time
        c = s["w"][lo:lo + 16384].to(torch.int16)
        c = torch.stack((c & 15, c >> 4), 2).reshape(-1, k)
        e, f = (c >> 1) & 3, (c & 1).double()
        v = torch.where(e == 0, f / 2, (2 + f) * torch.exp2(e.double() - 2))
        group = torch.arange(k, device=x.device) // case["kblock"]
        v = torch.where(c >= 8, -v, v) * torch.exp2(s["sf"][lo:lo + 16384].double() - 127)[:, group]
        parts.append(x @ v.t().contiguous())
    return torch.cat(parts, 1)
