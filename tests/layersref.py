"""Plain 64-bit forms of the feed-forward layer's operators, from their
definitions, and error bounds of the kernels' arithmetic, for the GPU tests
(torch, no code shared with the kernels).

u = 2^-24 is half a step of fp32 relative to the value; a sum of n products in
fp32, in any order, is off by at most n u times the sum of their magnitudes
(a matrix instruction's products of 16-bit numbers are exact)."""
import math

import torch

from opsref import HALF, TINY, U

KIND = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "fp16"}
ACTS = ["silu", "gelu", "gelu_tanh", "relu"]
DEV = torch.device("cuda:0")


def rand(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def act(name, g):
    """(act(g), act'(g)) of float64 g."""
    if name == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * torch.sigmoid(-g))
    if name == "gelu":
        p = torch.special.erfc(-g / math.sqrt(2)) / 2
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        return g * (1 + t) / 2, (1 + t) / 2 + g / 2 * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    return g.clamp_min(0), (g > 0).double()


def act_error(name, g):
    """Relative to p = act(g) / g, how far the kernels' p may be off, in steps
    of fp32 (2 u): exp(z) is off by |z| steps (its argument's rounding) and
    three operations follow; gelu's erfc moves by g^2 times its argument's
    rounding, and is itself good to 16 steps; gelu_tanh's |z| = 1.6 |g| +
    0.0714 |g|^3 is off by four roundings before its exp."""
    a = g.abs()
    if name == "silu":
        steps = a + 6
    elif name == "gelu":
        steps = a * a + 24
    elif name == "gelu_tanh":
        steps = 5 * (1.6 * a + 0.0714 * a ** 3).clamp_max(200) + 6
    else:
        return torch.zeros_like(g)
    return steps * 2 * U


def half(want, bound, dtype):
    """The rounding of a value within `bound` of `want` to dtype."""
    k = KIND[dtype]
    return bound + HALF[k] * (want.abs() + bound) + TINY[k]


def glu(x, wg, wu, name):
    """(h, g, u and their bounds before the results' rounding)."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    n = x.shape[1] + 1
    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = n * U * (x.abs() @ wg.abs().t()), n * U * (x.abs() @ wu.abs().t())
    value, _ = act(name, g)
    # |act'| is at most 1.13; p's own error on |g|; the last product's rounding
    ea = 1.13 * eg + act_error(name, g) * (value.abs() + eg) + 2.0 ** -126
    h = value * u
    eh = ea * (u.abs() + eu) + (value.abs() + ea) * eu + U * h.abs()
    return (h, g, u), (eh, eg, eu)


def glu_parts(dh, g, u, name):
    """(dg, du) and their bounds before rounding."""
    dh, g, u = dh.double(), g.double(), u.double()
    value, slope = act(name, g)
    rel = act_error(name, g)
    # slope = p + g p (1 - p) z': p's error on each factor, 1 - p off by a step, five operations; |g p z'| where
    # 1 - p counts is below 2 |value| max(1, z')
    z = {"silu": torch.ones_like(g), "gelu_tanh": 1.6 + 0.22 * g * g}.get(name, torch.ones_like(g))
    on = (g.abs() < 64) if name == "gelu_tanh" else torch.ones_like(g, dtype=torch.bool)
    ev = (rel + 4 * U) * value.abs() + 2.0 ** -126
    es = (rel * 3 + 12 * U) * (1 + value.abs() * torch.where(on, z, 0)) + 2.0 ** -126
    if name == "gelu":
        # the density e^(-g^2/2): its argument's rounding is g^2 / 2 steps
        es = es + (g * g + 8) * 2 * U * g.abs() * torch.exp(-g * g / 2)
    if name == "relu":
        ev, es = 0 * ev, 0 * es
    dg, du = dh * u * slope, dh * value
    return (dg, du), ((dh * u).abs() * es + 2 * U * dg.abs(), dh.abs() * ev + U * du.abs())


def glu_backward(dh, g, u, x, wg, wu, name):
    """((dx, dwg, dwu), bounds before the results' rounding): dg and du are
    rounded to x's type, which their products' bounds carry."""
    t = x.dtype
    (dg, du), (eg, eu) = glu_parts(dh, g, u, name)
    eg, eu = half(dg, eg, t), half(du, eu, t)
    x, wg, wu = x.double(), wg.double(), wu.double()

    def product(pairs, n):
        v = sum(a @ b for a, _, b in pairs)
        e = sum(ea @ b.abs() + (n + 1) * U * ((a.abs() + ea) @ b.abs()) for a, ea, b in pairs)
        return v, e

    dx = product([(dg, eg, wg), (du, eu, wu)], 2 * wg.shape[0])
    dwg = product([(dg.t().contiguous(), eg.t().contiguous(), x)], x.shape[0])
    dwu = product([(du.t().contiguous(), eu.t().contiguous(), x)], x.shape[0])
    return (dx[0], dwg[0], dwu[0]), (dx[1], dwg[1], dwu[1])


def within(got, want, bound, what=""):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), "%s: %d of %d off, worst %.3g against %.3g" % (
        what, int(bad.sum()), bad.numel(), float(off[bad].max()), float(bound[bad].max()))


def quantize(x):
    """(codes, scales) of float32/16 x by the definition: the scale in fp32,
    codes of the exact quotient (a quotient of two fp32 numbers that is no tie
    is at least 2^-33 from one, relative: float64 shows the side)."""
    # (divided in 64 bits and rounded: the division of fp32 by a plain number is a product with its rounded inverse
    # in torch; 53 bits are over twice 24 plus two, so the second rounding gives what one would)
    top = x.double().abs().amax(1) if x.shape[1] else x.new_zeros(x.shape[0], dtype=torch.float64)
    scale = (top / 127).float().clamp_min(2.0 ** -126)
    return torch.round(x.double() / scale.double()[:, None]).to(torch.int8), scale
