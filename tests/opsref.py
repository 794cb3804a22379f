"""Plain 64-bit forms of the operators around the block-scaled products, from
their definitions, for the GPU tests (numpy, no code shared with the
kernels), and the error bounds those tests use.

u = 2^-24 is half a step of fp32 relative to the value; a sum of n terms in
fp32, in any order, is off by at most (n - 1) u times the sum of the terms'
magnitudes, and by at most the longest chain of additions in place of n - 1.
"""
import numpy as np

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "f32": 2.0 ** -24}           # half a step, relative
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "f32": 2.0 ** -150}        # half a step of the subnormals
SIG = {"bf16": (7, -126), "fp16": (10, -14), "f32": (23, -126)}


def round_to(v, kind):
    """float64 v rounded to nearest even in the type (values in its range)."""
    bits, low = SIG[kind]
    _, p = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(p - 1, low) - bits)
    return np.rint(v / step) * step


def e4m3(codes):
    """Values of e4m3 codes (uint8) in float64."""
    c = codes.astype(np.int64)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, np.ldexp(f.astype(np.float64), -9), np.ldexp(8.0 + f, e - 10))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def dequant(q, sf):
    """float64 values of block-scaled rows (uint8 codes and scales)."""
    return e4m3(q) * np.repeat(np.ldexp(1.0, sf.astype(np.int64) - 127), 32, axis=1)


def quantize(x):
    """(element values in units of the block's scale, scale codes) of the rows of float64 x."""
    rows, n = x.shape
    b = x.reshape(rows, n // 32, 32)
    fin = np.where(np.isfinite(b), np.abs(b), 0.0).max(axis=2)
    f, p = np.frexp(fin)                               # fin = f * 2^p, f in [0.5, 1)
    e = np.where(fin == 0, -127, np.maximum(p - 9 + (f > 0.875), -127))
    v = b / np.ldexp(1.0, e)[:, :, None]
    v = np.where(np.isfinite(v), v, np.nan)
    _, pv = np.frexp(np.where(np.isnan(v), 0.0, v))
    step = np.ldexp(1.0, np.maximum(pv - 1, -6) - 3)
    return (np.rint(v / step) * step).reshape(rows, n), e + 127


E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def fp4_weights(w, sf, kblock):
    """float64 values of (N, K/2) bytes with their group scales."""
    v = np.stack((E2M1[w & 15], E2M1[w >> 4]), axis=2).reshape(w.shape[0], -1)
    scale = np.ldexp(1.0, sf.astype(np.int64) - 127)
    return v * scale[:, np.arange(v.shape[1]) // kblock]


def norm(h, w, eps):
    """(y, rstd) of float64 rows h."""
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * w * rstd[:, None], rstd


def rstd_bound(n):
    """Relative: the longest chain of additions of a row's sum (n / 64 a lane
    at most, and 32 to join them), halved by the square root, and four
    roundings (mean, eps, root, division)."""
    return ((n / 64 + 32) / 2 + 4) * U


def norm_backward(dy, h, w, rstd, dh):
    """(dx, dw) and, for the bounds, |rstd g|, |rstd u| mean|g u| and sum|dy u|."""
    u, g = h * rstd[:, None], dy * w
    m = (g * u).mean(axis=1, keepdims=True)
    a = np.abs(g * u).mean(axis=1, keepdims=True)
    dx = rstd[:, None] * (g - u * m) + dh
    return dx, (dy * u).sum(axis=0), rstd[:, None] * np.abs(g), rstd[:, None] * np.abs(u) * a, np.abs(dy * u).sum(axis=0)
