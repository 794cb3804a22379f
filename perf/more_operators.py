"""Operators of a feed-forward layer's linear parts, as timed and compared cases.

Five operators: the gated block of a feed-forward layer (``glu``) with its backward pass (``glubwd``), what makes an
8-bit integer operand (``quant``) and the product of two of them (``int8``), and the clipping of a model's gradients
by their common norm (``clip``).  With ``own`` false each runs in its plain form, elementary torch operations in 32
bits; with ``own`` true through the package's entry points.

Definitions:
  glu     g = x wg^T, u = x wu^T, h = act(g) * u; g and u are given out too where a backward pass will read them
  glubwd  du = dh * act(g), dg = dh * u * act'(g);  dx = dg wg + du wu, dwg = dg^T x, dwu = du^T x, the weights'
          gradients added to those of earlier micro-batches where there are any
  quant   s = max(max|x| / 127, 2^-126) of a row, rounded to fp32; q = x / s rounded to nearest even
  int8    d[m, n] = c[m, n] + sa[m] * sb[n] * sum over k of a[m, k] * b[n, k]
  clip    norm = sqrt(sum of all gradients' squares); every gradient times min(1, top / (norm + 1e-6))
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "f32": 4}
MOST = 8192 * 14336 * 4096          # multiplications of the largest product


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one token of a decode step through the gated block
        dict(name="glu_token_bf16", op="glu", m=1, f=14336, k=4096, type="bf16", act="silu", keep=False),
        # a batch of 16 sequences, one token each, another activation
        dict(name="glu_batch16_fp16", op="glu", m=16, f=14336, k=5120, type="fp16", act="gelu_tanh", keep=False),
        # a training batch: g and u are kept for the backward pass
        dict(name="glu_train_bf16", op="glu", m=8192, f=14336, k=4096, type="bf16", act="silu", keep=True),
        # the same batch's backward pass
        dict(name="glubwd_batch_bf16", op="glubwd", m=8192, f=14336, k=4096, type="bf16", act="silu", acc=False),
        # a small layer with odd sizes, added to the gradients of earlier micro-batches
        dict(name="glubwd_ragged_fp16", op="glubwd", m=1001, f=2731, k=1003, type="fp16", act="gelu", acc=True),
        # a prompt's activation on its way into an 8-bit product
        dict(name="quant_prompt_bf16", op="quant", rows=8192, n=14336, type="bf16"),
        # a short, ragged one
        dict(name="quant_short_fp16", op="quant", rows=77, n=4100, type="fp16"),
        # one token through the projection back
        dict(name="int8_token", op="int8", m=1, n=4096, k=14336, out="bf16", acc=False),
        # a few dozen rows, odd sizes, onto the residual stream
        dict(name="int8_ragged", op="int8", m=77, n=4099, k=4100, out="f32", acc=True),
        # a prompt
        dict(name="int8_prompt", op="int8", m=8192, n=14336, k=4096, out="bf16", acc=False),
        # the gradients of one small layer, some in fp32
        dict(name="clip_layer", op="clip", layers=1, d=512, f=1376, type="mixed", top=1.0),
        # the gradients of six large layers, 1.3 billion weights
        dict(name="clip_model_bf16", op="clip", layers=6, d=4096, f=14336, type="bf16", top=1.0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _near(rng, n):
    """n, or two times in three the multiple of 8 or of 128 next to it: sizes as models have them, and any."""
    step = rng.choice([1, 8, 128])
    return max(step, step * round(n / step))


def draw(rng):
    op = rng.choice(["glu", "glubwd", "quant", "int8", "clip"])
    kind = rng.choice(["bf16", "fp16"])
    if op in ("glu", "glubwd"):
        f, k = _near(rng, _log(rng, 64, 14336)), _near(rng, _log(rng, 64, 4096))
        m = max(1, min(_log(rng, 1, 8192), MOST // (f * k)))
        case = dict(op=op, m=m, f=f, k=k, type=kind, act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]))
        return dict(case, keep=rng.random() < 0.5) if op == "glu" else dict(case, acc=rng.random() < 0.5)
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 8192), n=_near(rng, _log(rng, 16, 14336)), type=rng.choice(list(TYPES)))
    if op == "int8":
        n, k = _near(rng, _log(rng, 64, 32768)), _near(rng, _log(rng, 64, 14336))
        return dict(op=op, m=max(1, min(_log(rng, 1, 8192), MOST // (n * k))), n=n, k=k,
                    out=rng.choice(list(TYPES)), acc=rng.random() < 0.4)
    return dict(op=op, layers=_log(rng, 1, 6), d=_log(rng, 33, 4096), f=_log(rng, 65, 14336),
                type=rng.choice(["bf16", "fp16", "f32", "mixed"]) if rng.random() < 0.5 else "bf16",
                top=rng.choice([0.5, 1.0, 1e9]))


def _shapes(case):
    """The shapes of a model's gradients: four projections of attention, three of the block, two norms a layer."""
    d, f = case["d"], case["f"]
    return [(d, d), (d // 4 + 1, d), (d // 4 + 1, d), (d, d), (f, d), (f, d), (d, f), (d,), (d,)] * case["layers"]


def _type_of(case, i):
    return (("bf16", "f32", "fp16")[i % 3] if case["type"] == "mixed" else case["type"])


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

    if op in ("glu", "glubwd"):
        m, f, k, t = case["m"], case["f"], case["k"], TYPES[case["type"]]
        s["x"] = noise(m, k).to(t)                       # (behind a norm)
        s["wg"], s["wu"] = (noise(f, k) * k ** -0.5).to(t), (noise(f, k) * k ** -0.5).to(t)
        if op == "glu":
            s["h"] = room(m, f, dtype=t)
            s["g"], s["u"] = (room(m, f, dtype=t), room(m, f, dtype=t)) if case["keep"] else (None, None)
            return s
        s["g"], s["u"], s["dh"] = noise(m, f).to(t), noise(m, f).to(t), noise(m, f).to(t)
        if case["acc"]:
            s["cg"], s["cu"] = noise(f, k).to(t), noise(f, k).to(t)
        s["dx"], s["dwg"], s["dwu"] = room(m, k, dtype=t), room(f, k, dtype=t), room(f, k, dtype=t)
        if torch.cuda.is_available():                    # kept for the program's life: enough for the largest batch
            s["ws"] = room(8 * (m + 128) * (f + 128) + 2 * (m + 128) * (k + 128) + 4 * (f + 128) * (k + 128) + (1 << 20),
                           dtype=torch.uint8)
        return s
    if op == "quant":
        rows, n = case["rows"], case["n"]
        s["x"] = _activations(g, rows, n, TYPES[case["type"]])
        s["q"], s["s"] = room(rows, n, dtype=torch.int8), room(rows, dtype=torch.float32)
        return s
    if op == "int8":
        m, n, k, t = case["m"], case["n"], case["k"], TYPES[case["out"]]

        def codes(rows):
            return (noise(rows, k) * 30).round().clamp(-127, 127).to(torch.int8)

        s["a"], s["b"] = codes(m), codes(n)
        s["sa"] = 0.03 * (1 + torch.rand(m, generator=g, device=dev))
        s["sb"] = 0.001 * (1 + torch.rand(n, generator=g, device=dev))
        s["c"] = noise(m, n).to(t) if case["acc"] else None
        s["d"] = room(m, n, dtype=t)
        return s
    s["grads"] = [(noise(*shape) * 0.01).to(TYPES[_type_of(case, i)]) for i, shape in enumerate(_shapes(case))]
    s["out"] = [torch.empty_like(t) for t in s["grads"]]
    return s


# ---- plain forms and calls --------------------------------------------------

R2, RPI = 0.7071067811865476, 0.7978845608028654       # sqrt(1/2), sqrt(2/pi)


def _act(name, g):
    if name == "silu":
        return g / (1 + torch.exp(-g))
    if name == "relu":
        return g.clamp_min(0)
    if name == "gelu":
        return 0.5 * g * (1 + torch.erf(g * R2))
    return 0.5 * g * (1 + torch.tanh(RPI * (g + 0.044715 * g * g * g)))


def _slope(name, g):
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    if name == "relu":
        return (g > 0).to(g.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(g * R2)) + g * torch.exp(-0.5 * g * g) * (0.5 * RPI)
    t = torch.tanh(RPI * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * RPI * (1 + 3 * 0.044715 * g * g)


def _glu(s):
    x, t = s["x"].float(), s["x"].dtype
    g, u = torch.mm(x, s["wg"].float().t()), torch.mm(x, s["wu"].float().t())
    h = (_act(s["act"], g) * u).to(t)
    return (h, g.to(t), u.to(t)) if s["keep"] else h


def _glubwd(s):
    t = s["x"].dtype
    g, dh, x = s["g"].float(), s["dh"].float(), s["x"].float()
    du = dh * _act(s["act"], g)
    dg = dh * s["u"].float() * _slope(s["act"], g)
    dx = torch.mm(dg, s["wg"].float()) + torch.mm(du, s["wu"].float())
    dwg, dwu = torch.mm(dg.t(), x), torch.mm(du.t(), x)
    if s["acc"]:
        dwg, dwu = dwg + s["cg"].float(), dwu + s["cu"].float()
    return dx.to(t), dwg.to(t), dwu.to(t)


def _quant(s):
    x = s["x"].float()
    # (in 64 bits: the nearest of two codes is a matter of the last bit at a border, and torch divides fp32 by a
    # plain number as a product with its rounded inverse)
    scale = (x.abs().amax(1).double() / 127).float().clamp_min(2.0 ** -126)
    return torch.round(x.double() / scale.double()[:, None]).to(torch.int8), scale


def _int8(s):
    d = torch.mm(s["a"].float(), s["b"].float().t()) * (s["sa"][:, None] * s["sb"])
    if s["c"] is not None:
        d = d + s["c"].float()
    return d.to(s["d"].dtype)


def _clip(s):
    norm = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt()
    by = (s["top"] / (norm + 1e-6)).clamp_max(1)
    return norm, [(t.float() * by).to(t.dtype) for t in s["grads"]]


def run(state):
    s, op = state, state["op"]
    if not own:
        return {"glu": _glu, "glubwd": _glubwd, "quant": _quant, "int8": _int8, "clip": _clip}[op](s)
    import tiled_dense_gemm_tile_amd as tg
    if op == "glu":
        return tg.gemm_glu(s["x"], s["wg"], s["wu"], act=s["act"], H=s["h"], G=s["g"], U=s["u"])
    if op == "glubwd":
        cg, cu = (s["cg"], s["cu"]) if s["acc"] else (None, None)
        return tg.gemm_glu_backward(s["dh"], s["g"], s["u"], s["x"], s["wg"], s["wu"], act=s["act"], Cg=cg, Cu=cu,
                                    dX=s["dx"], dWg=s["dwg"], dWu=s["dwu"], workspace=s["ws"])
    if op == "quant":
        return tg.int8_quantize(s["x"], Q=s["q"], S=s["s"])
    if op == "int8":
        return tg.gemm_int8(s["a"], s["sa"], s["b"], s["sb"], C=s["c"], D=s["d"], out_dtype=s["d"].dtype)
    return tg.clip_grads(s["grads"], s["top"], out=s["out"]), s["out"]


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    op = case["op"]
    if op in ("glu", "glubwd"):
        m, f, k = case["m"], case["f"], case["k"]
        if op == "glu":
            return {"bytes": 2 * (m * k + 2 * f * k + m * f * (3 if case["keep"] else 1)), "flops": 4 * m * f * k}
        return {"bytes": 2 * (3 * m * f + 2 * m * k + (6 if case["acc"] else 4) * f * k), "flops": 8 * m * f * k}
    if op == "quant":
        e = case["rows"] * case["n"]
        return {"bytes": e * SIZE[case["type"]] + e + 4 * case["rows"], "flops": 3 * e}
    if op == "int8":
        m, n, k, z = case["m"], case["n"], case["k"], SIZE[case["out"]]
        return {"bytes": m * k + n * k + 4 * (m + n) + m * n * z * (2 if case["acc"] else 1), "flops": 2 * m * n * k}
    sizes = [(math.prod(shape), SIZE[_type_of(case, i)]) for i, shape in enumerate(_shapes(case))]
    return {"bytes": sum(2 * e * z for e, z in sizes), "flops": sum(3 * e for e, _ in sizes)}


# ---- the definitions in 64 bits ---------------------------------------------

def _gate(name, g):
    """(act(g), act'(g)) in float64, from the logistic and normal distribution functions."""
    if name == "relu":
        on = (g > 0).double()
        return g * on, on
    if name == "gelu":
        below = torch.special.erfc(-g / math.sqrt(2)) / 2
        return g * below, below + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * torch.sigmoid(-g)
    inner = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    p = torch.sigmoid(inner)                             # (1 + tanh(z)) / 2 = sigmoid(2 z)
    return g * p, p + g * p * torch.sigmoid(-inner) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "glu":
        x = s["x"].double()
        g, u = x @ s["wg"].double().t(), x @ s["wu"].double().t()
        h = _gate(case["act"], g)[0] * u
        return (h, g, u) if case["keep"] else h
    if op == "glubwd":
        x, dh = s["x"].double(), s["dh"].double()
        value, slope = _gate(case["act"], s["g"].double())
        both = torch.cat((dh * s["u"].double() * slope, dh * value), 1)
        dx = both @ torch.cat((s["wg"].double(), s["wu"].double()))
        dw = both.t().contiguous() @ x
        dwg, dwu = dw[:case["f"]], dw[case["f"]:]
        return (dx, dwg + s["cg"].double(), dwu + s["cu"].double()) if case["acc"] else (dx, dwg, dwu)
    if op == "quant":
        x = s["x"].double()
        scale = torch.maximum(x.abs().max(1).values / 127, torch.tensor(2.0 ** -126, device=x.device))
        return torch.round(x / scale.float().double()[:, None]), scale
    if op == "int8":
        d = (s["a"].double() @ s["b"].double().t()) * s["sb"].double() * s["sa"].double()[:, None]
        return d if s["c"] is None else d + s["c"].double()
    norm = math.sqrt(sum(float(torch.dot(t.double().flatten(), t.double().flatten())) for t in s["grads"]))
    by = min(1.0, case["top"] / (norm + 1e-6))
    return torch.tensor(norm, dtype=torch.float64), [t.double() * by for t in s["grads"]]
