"""The feed-forward layer's operators against plain 64-bit forms: the gated
block and its gradients, 8-bit integer products, gradient clipping."""
import math

import pytest
import torch

import layersref as ref
import tiled_dense_gemm_tile_amd as tg
from layersref import DEV, KIND, U, act, half, rand, within
from opsref import HALF, TINY

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def padded(t, ld, fill=float("nan")):
    """t as a view of a wider matrix whose other columns hold `fill`."""
    w = torch.full((t.shape[0] + 1, ld), fill, dtype=t.dtype, device=t.device)
    w[:t.shape[0], :t.shape[1]] = t
    return w[:t.shape[0], :t.shape[1]]


def check_glu(x, wg, wu, name, keep=True, **out):
    got = tg.gemm_glu(x, wg, wu, act=name, keep=keep, **out)
    want, bound = ref.glu(x, wg, wu, name)
    for v, w, b, n in zip(got if keep else (got,), want, bound, "hgu"):
        within(v, w, half(w, b, x.dtype), "%s %s" % (name, n))


# few rows, one tile, several tiles, odd sizes, K inside a 16-byte chunk, K past one tile, K = 1
GLU_SIZES = [(1, 64, 64), (1, 1, 1), (2, 17, 31), (16, 48, 1000), (17, 100, 130), (32, 130, 513), (33, 32, 64),
             (64, 96, 128), (77, 131, 200), (130, 333, 77), (200, 640, 1), (300, 1000, 264), (512, 2304, 192)]


@pytest.mark.parametrize("m,f,k", GLU_SIZES)
@pytest.mark.parametrize("dtype", [BF, FP], ids=KIND.get)
def test_glu(m, f, k, dtype):
    x, wg, wu = rand(1, m, k, dtype=dtype), rand(2, f, k, dtype=dtype, scale=k ** -0.5), rand(3, f, k, dtype=dtype, scale=k ** -0.5)
    check_glu(x, wg, wu, "silu")


@pytest.mark.parametrize("m", [1, 40, 300])
@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("dtype", [BF, FP], ids=KIND.get)
def test_glu_activations(m, name, dtype):
    """Arguments over the activations' whole course, far tails among them."""
    x, wg, wu = rand(4, m, 96, dtype=dtype), rand(5, 80, 96, dtype=dtype, scale=0.6), rand(6, 80, 96, dtype=dtype, scale=0.1)
    check_glu(x, wg, wu, name)


@pytest.mark.parametrize("m", [3, 100, 400])
@pytest.mark.parametrize("dtype", [BF, FP], ids=KIND.get)
def test_glu_strides(m, dtype):
    """Leading dimensions that keep rows on and off 16 bytes, NaN around every operand; results only where they belong."""
    f, k = 136, 152
    for ldx, ldw, ldh, shift in ((160, 168, 144, 0), (153, 155, 137, 1), (152, 154, 139, 3)):
        x, wg, wu = (padded(rand(i, r, k, dtype=dtype, scale=0.3), ld + shift)[:, :]
                     for i, r, ld in ((1, m, ldx), (2, f, ldw), (3, f, ldw + 3)))
        outs = [padded(torch.zeros(m, f, dtype=dtype, device=DEV), ldh + i, 7.0) for i in range(3)]
        check_glu(x, wg, wu, "gelu", H=outs[0], G=outs[1], U=outs[2])
        for i, o in enumerate(outs):
            whole = o.as_strided((m + 1, ldh + i), (ldh + i, 1))
            assert bool((whole[:, f:] == 7).all()) and bool((whole[m] == 7).all())


def test_glu_base_off_16_bytes():
    """Operands that start one element into an allocation."""
    for m in (5, 200):
        buf = [rand(i, r * 128 + 1)[1:].reshape(r, 128) for i, r in ((1, m), (2, 160), (3, 160))]
        check_glu(*buf, "silu")


def test_glu_halves_of_one_weight():
    w, x = rand(1, 2 * 200, 128, scale=0.1), rand(2, 70, 128)
    check_glu(x, w[:200], w[200:], "silu", keep=False)
    both = rand(3, 200, 256, scale=0.1)                # side by side in a row
    check_glu(x, both[:, :128], both[:, 128:], "silu", keep=False)
    assert torch.equal(tg.gemm_glu(x, w[:200], w[200:]), tg.gemm_glu(x, w[:200].clone(), w[200:].clone()))


@pytest.mark.parametrize("m", [4, 64, 300])
def test_glu_keeps_one_of_both(m):
    x, wg, wu = rand(1, m, 128), rand(2, 96, 128), rand(3, 96, 128)
    h, g, u = tg.gemm_glu(x, wg, wu, keep=True)
    G = torch.empty_like(g)
    h1, g1, u1 = tg.gemm_glu(x, wg, wu, G=G)
    assert u1 is None and torch.equal(h, h1) and torch.equal(g, g1)
    assert torch.equal(h, tg.gemm_glu(x, wg, wu))


def test_glu_empty():
    w = rand(1, 40, 64)
    assert tg.gemm_glu(rand(2, 0, 64), w, w).shape == (0, 40)
    assert tg.gemm_glu(rand(2, 5, 64), w[:0], w[:0]).shape == (5, 0)
    for m in (5, 50):
        assert bool((tg.gemm_glu(rand(2, m, 64)[:, :0], w[:, :0], w[:, :0]) == 0).all())


@pytest.mark.parametrize("m", [2, 70])
def test_glu_not_finite(m):
    """An infinity or a NaN in one row stays in that row, one in a weight row in that column."""
    x, wg, wu = rand(1, m, 130), rand(2, 60, 130), rand(3, 60, 130)
    clean = tg.gemm_glu(x, wg, wu)
    for v in (float("inf"), float("nan")):
        y = x.clone()
        y[1, 129] = v
        got = tg.gemm_glu(y, wg, wu)
        assert torch.equal(got[0], clean[0]) and torch.equal(got[2:], clean[2:])
        assert not bool(got[1].isfinite().all())
        w = wu.clone()
        w[7, 0] = v
        got = tg.gemm_glu(x, wg, w)
        assert not bool(got[:, 7].isfinite().any())
        got[:, 7] = clean[:, 7]
        assert torch.equal(got, clean)


# ---- gradients of the gated block ---------------------------------------------------

def check_backward(m, f, k, dtype, name="silu", acc=False, grad=None, seed=0, scale=1.0):
    grad = grad or dtype
    dh, g, u = (rand(seed + i, m, f, dtype=dtype) for i in (1, 2, 3))
    g = g * scale
    x, wg, wu = rand(seed + 4, m, k, dtype=dtype), rand(seed + 5, f, k, dtype=dtype, scale=0.2), rand(seed + 6, f, k, dtype=dtype, scale=0.2)
    cg, cu = (rand(seed + 7, f, k, dtype=grad), rand(seed + 8, f, k, dtype=grad)) if acc else (None, None)
    got = tg.gemm_glu_backward(dh, g, u, x, wg, wu, act=name, Cg=cg, Cu=cu, grad_dtype=grad)
    want, bound = ref.glu_backward(dh, g, u, x, wg, wu, name)
    for v, w, b, n, c, t in zip(got, want, bound, ("dx", "dwg", "dwu"), (None, cg, cu), (dtype, grad, grad)):
        if c is not None:
            w = w + c.double()
            b = b + U * (w.abs() + b)
        assert v.dtype == t
        within(v, w, half(w, b, t), "%s %s" % (name, n))


@pytest.mark.parametrize("m,f,k", [(1, 1, 1), (1, 64, 64), (3, 17, 31), (64, 64, 64), (65, 130, 67), (200, 100, 333),
                                   (513, 72, 200), (128, 700, 640), (700, 1100, 520)])
@pytest.mark.parametrize("dtype,grad", [(BF, BF), (BF, F32), (FP, FP), (FP, F32)])
def test_glu_backward(m, f, k, dtype, grad):
    check_backward(m, f, k, dtype, grad=grad, acc=m % 2 == 1)


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("dtype", [BF, FP], ids=KIND.get)
def test_glu_backward_activations(name, dtype):
    check_backward(90, 110, 70, dtype, name, scale=4.0)


def test_glu_backward_strides():
    m, f, k = 70, 90, 110
    dh, g, u = (padded(rand(i, m, f), 91 + i) for i in range(3))
    x, wg, wu = padded(rand(4, m, k), 111), padded(rand(5, f, k), 113), padded(rand(6, f, k), 120)
    want = tg.gemm_glu_backward(*(t.contiguous() for t in (dh, g, u, x, wg, wu)))
    outs = [padded(torch.zeros(r, k, device=DEV, dtype=BF), ld, 7.0) for r, ld in ((m, 111), (f, 112), (f, 115))]
    tg.gemm_glu_backward(dh, g, u, x, wg, wu, dX=outs[0], dWg=outs[1], dWu=outs[2])
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
        whole = o.as_strided((o.shape[0] + 1, o.stride(0)), (o.stride(0), 1))
        assert bool((whole[:, k:] == 7).all()) and bool((whole[-1] == 7).all())


def test_glu_backward_in_place_and_parts():
    """Accumulation in place, into the halves of one tensor, and each gradient alone: the same bits."""
    m, f, k = 130, 96, 72
    a = [rand(i, m, f) for i in range(3)] + [rand(3, m, k), rand(4, f, k), rand(5, f, k)]
    c = rand(6, 2 * f, k, dtype=F32)
    want = tg.gemm_glu_backward(*a, Cg=c[:f], Cu=c[f:], grad_dtype=F32)
    d = c.clone()
    got = tg.gemm_glu_backward(*a, Cg=d[:f], Cu=d[f:], dWg=d[:f], dWu=d[f:])
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    dx, none, none2 = tg.gemm_glu_backward(*a, weight_grad=False)
    assert none is None and none2 is None and torch.equal(dx, want[0])
    none, dwg, dwu = tg.gemm_glu_backward(*a, Cg=c[:f], Cu=c[f:], grad_dtype=F32, input_grad=False)
    assert none is None and torch.equal(dwg, want[1]) and torch.equal(dwu, want[2])


def test_glu_backward_empty():
    w, c = rand(1, 40, 64), rand(2, 40, 64)
    e, x = rand(3, 0, 40), rand(3, 0, 64)
    dx, dwg, dwu = tg.gemm_glu_backward(e, e, e, x, w, w, Cg=c, Cu=c)
    assert dx.shape == (0, 64) and torch.equal(dwg, c) and torch.equal(dwu, c)
    assert bool((tg.gemm_glu_backward(e, e, e, x, w, w)[1] == 0).all())
    e, x = rand(3, 9, 0), rand(3, 9, 64)
    dx, dwg, dwu = tg.gemm_glu_backward(e, e, e, x, w[:0], w[:0])
    assert bool((dx == 0).all()) and dwg.shape == (0, 64)


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_glu_gradient_is_the_slope(name):
    """Gradients against central differences of the definition in 64 bits.  A step of e = 2^-10 is off by e^2 / 6
    times a third derivative (below 2 |dh u| |x|^3 here), far under the 16-bit results' half step, which with the
    operands' own rounding is the bound."""
    m, f, k = 24, 40, 16
    x, wg, wu = rand(1, m, k, dtype=FP), rand(2, f, k, dtype=FP, scale=0.25), rand(3, f, k, dtype=FP, scale=0.25)
    dh = rand(4, m, f, dtype=FP)
    _, g, u = tg.gemm_glu(x, wg, wu, act=name, keep=True)
    dx, dwg, dwu = tg.gemm_glu_backward(dh, g, u, x, wg, wu, act=name, grad_dtype=F32)

    def loss(x, wg, wu):
        return ((act(name, x @ wg.t())[0] * (x @ wu.t())) * dh.double()).sum()

    a = [t.double() for t in (x, wg, wu)]
    gen = torch.Generator(DEV).manual_seed(9)
    for i, grad in enumerate((dx, dwg, dwu)):
        d = torch.randn(a[i].shape, generator=gen, device=DEV, dtype=torch.float64)
        d = d / d.norm()
        e = 2.0 ** -10
        up = loss(*(t + e * d if j == i else t for j, t in enumerate(a)))
        down = loss(*(t - e * d if j == i else t for j, t in enumerate(a)))
        # g, u, dg, du and dx are each rounded by half a step of fp16: 5 * 2^-11 of the terms' norm, which is at
        # most that of the gradient times a few
        assert abs(float((up - down) / (2 * e) - (grad.double() * d).sum())) <= 5 * HALF["fp16"] * 4 * float(grad.double().norm())


# ---- 8-bit integers -----------------------------------------------------------------

@pytest.mark.parametrize("rows,n", [(1, 1), (1, 14336), (3, 7), (5, 64), (70, 511), (4, 513), (9, 2048), (33, 4100), (2, 8200),
                                    (3, 16385), (2, 40000), (1000, 96), (1500, 96), (1100, 700), (1024, 1500),
                                    (1030, 3001), (1025, 5000), (1025, 9001), (1024, 17000), (7, 1200), (5, 3000), (1, 20000)])
@pytest.mark.parametrize("dtype", [F32, BF, FP], ids=KIND.get)
def test_quantize(rows, n, dtype):
    x = rand(rows + n, rows, n, dtype=dtype)
    q, s = tg.int8_quantize(x)
    wq, ws = ref.quantize(x)
    assert torch.equal(s, ws) and torch.equal(q, wq)
    # rows at odd places, results only where they belong
    big = padded(x, n + 3)
    out = torch.full((rows, n + 5), 99, dtype=torch.int8, device=DEV)
    tg.int8_quantize(big, Q=out[:, 1:n + 1])
    assert torch.equal(out[:, 1:n + 1], wq) and bool((out[:, 0] == 99).all()) and bool((out[:, n + 1:] == 99).all())


def test_quantize_ties_go_to_even():
    """Every border k + 1/2 of a scale of 1 and its neighbours, and borders of scales that are no powers of two."""
    h = torch.arange(-126, 127, device=DEV, dtype=torch.float32) + 0.5
    row = torch.cat([torch.tensor([127.0], device=DEV), h, torch.nextafter(h, h + 1), torch.nextafter(h, h - 1)])
    q, s = tg.int8_quantize(row[None])
    assert float(s) == 1.0 and torch.equal(q[0].double(), torch.round(row.double()))
    x = rand(1, 64, 4096, dtype=F32)
    scale = ref.quantize(x)[1]
    k = torch.randint(-126, 126, (64, 4095), device=DEV) + 0.5
    near = (k * scale[:, None]).float()
    for to in (near, torch.nextafter(near, near + 1), torch.nextafter(near, near - 1)):
        y = torch.cat([x.abs().amax(1, keepdim=True), to], 1)
        q, s = tg.int8_quantize(y)
        wq, ws = ref.quantize(y)
        assert torch.equal(s, ws) and torch.equal(q, wq)


def test_quantize_extremes():
    """Zeros, subnormals, the largest numbers, rows that are not finite."""
    x = torch.zeros(8, 300, device=DEV)
    x[1, 7] = 2.0 ** -149
    x[2, 5] = -3.4e38
    x[3] = 2.0 ** -126
    x[4, 299] = float("inf")
    x[5, 0] = float("nan")
    x[6] = torch.linspace(-1e-40, 1e-40, 300)
    q, s = tg.int8_quantize(x)
    ok = [0, 1, 2, 3, 6, 7]
    wq, ws = ref.quantize(x[ok])
    assert torch.equal(q[ok], wq) and torch.equal(s[ok], ws)
    assert bool(s[4:6].isnan().all()) and bool((q[4:6] == 0).all())
    q, s = tg.int8_quantize(x[:, :0])
    assert bool((s == 2.0 ** -126).all())


def check_int8(m, n, k, out=F32, c=None, lo=-128, pads=(0, 0, 0), seed=0):
    g = torch.Generator(DEV).manual_seed(seed + m * 7 + n * 3 + k)
    a = torch.randint(lo, 128, (m, k), generator=g, device=DEV, dtype=torch.int8)
    b = torch.randint(lo, 128, (n, k), generator=g, device=DEV, dtype=torch.int8)
    if any(pads):
        a, b = padded(a, k + pads[0], 77), padded(b, k + pads[1], 77)
    sa, sb = torch.rand(m, generator=g, device=DEV) + 0.5, torch.rand(n, generator=g, device=DEV) * 0.01
    C = None if c is None else rand(seed + 1, *((m, n) if c == "matrix" else (n,)), dtype=out)
    D = padded(torch.zeros(m, n, device=DEV, dtype=out), n + pads[2], 7.0) if pads[2] else None
    got = tg.gemm_int8(a, sa, b, sb, C=C, out_dtype=out, D=D)
    want = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()
    bound = 3 * U * want.abs()                         # the sum's, the scales' product's and the product's rounding
    if C is not None:
        want = want + C.double()
        bound = bound + U * (want.abs() + bound)
    within(got, want, half(want, bound, out) if out != F32 else bound + TINY["f32"], "int8 %s" % ((m, n, k),))
    if D is not None:
        whole = D.as_strided((m + 1, n + pads[2]), (n + pads[2], 1))
        assert bool((whole[:, n:] == 7).all()) and bool((whole[m] == 7).all())


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 64, 256), (1, 100, 4100), (2, 33, 15), (16, 200, 1000), (17, 64, 64),
                                   (32, 129, 777), (33, 70, 90), (64, 64, 128), (100, 130, 1030), (300, 500, 48), (600, 2500, 272)])
@pytest.mark.parametrize("out", [F32, BF, FP], ids=KIND.get)
def test_int8(m, n, k, out):
    check_int8(m, n, k, out)


@pytest.mark.parametrize("m", [3, 40, 300])
@pytest.mark.parametrize("c", ["matrix", "row"])
@pytest.mark.parametrize("out", [F32, BF, FP], ids=KIND.get)
def test_int8_c_and_strides(m, c, out):
    check_int8(m, 140, 160, out, c)
    check_int8(m, 140, 160, out, c, pads=(16, 32, 4))
    check_int8(m, 141, 163, out, c, pads=(1, 3, 5))


@pytest.mark.parametrize("m", [2, 50])
def test_int8_largest_sum(m):
    """K = 2^17 - 1 products of -128 with itself: just inside int32."""
    k = (1 << 17) - 1
    a, b = torch.full((m, k), -128, dtype=torch.int8, device=DEV), torch.full((20, k), -128, dtype=torch.int8, device=DEV)
    one, ones = torch.ones(m, device=DEV), torch.ones(20, device=DEV)
    want = torch.full((m, 20), float(k * 16384), device=DEV, dtype=torch.float64)
    within(tg.gemm_int8(a, one, b, ones), want, U * want)
    with pytest.raises(tg.GemmError):
        tg.gemm_int8(torch.zeros(1, k + 1, dtype=torch.int8, device=DEV), one[:1], torch.zeros(1, k + 1, dtype=torch.int8, device=DEV), ones[:1])


def test_int8_in_place_and_empty():
    a, sa = tg.int8_quantize(rand(1, 60, 128))
    b, sb = tg.int8_quantize(rand(2, 90, 128))
    c = rand(3, 60, 90, dtype=F32)
    want = tg.gemm_int8(a, sa, b, sb, C=c)
    d = c.clone()
    assert torch.equal(tg.gemm_int8(a, sa, b, sb, C=d, D=d), want)
    assert torch.equal(tg.gemm_int8(a[:, :0], sa, b[:, :0], sb, C=c), c)
    assert bool((tg.gemm_int8(a[:, :0], sa, b[:, :0], sb) == 0).all())
    assert tg.gemm_int8(a[:0], sa[:0], b, sb).shape == (0, 90)


def test_int8_rows_that_were_not_finite():
    x = rand(1, 40, 128)
    x[3, 5] = float("nan")
    a, sa = tg.int8_quantize(x)
    b, sb = tg.int8_quantize(rand(2, 50, 128))
    for rows in (slice(0, 8), slice(0, 40)):
        d = tg.gemm_int8(a[rows], sa[rows], b, sb)
        assert bool(d[3].isnan().all()) and bool(d[torch.arange(d.shape[0]) != 3].isfinite().all())


# ---- gradients' norm ----------------------------------------------------------------

def some_grads(seed, sizes, dtypes=(BF, F32, FP)):
    return [rand(seed + i, n, dtype=dtypes[i % len(dtypes)], scale=0.5) for i, n in enumerate(sizes)]


def norm64(grads):
    return math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))


SIZES = [[1], [0, 5], [8192], [8191, 8193, 3], [100000, 0, 1, 65536, 70001], list(range(1, 300))]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%dx" % len(s))
@pytest.mark.parametrize("top", [0.25, 1e9, 0.0])
def test_clip(sizes, top):
    grads = some_grads(1, sizes)
    want = norm64(grads)
    n = tg.grad_norm(grads)
    assert abs(float(n) - want) <= 2 * U * want + TINY["f32"]
    out = [torch.full_like(g, 7) for g in grads]
    n2 = tg.clip_grads(grads, top, out=out)
    assert torch.equal(n, n2)
    by = min(1.0, top / (want + 1e-6))
    copies = [g.clone() for g in grads]
    n3 = tg.clip_grads(copies, top)
    assert torch.equal(n, n3)
    for g, o, c in zip(grads, out, copies):
        assert torch.equal(o, c)
        w = g.double() * by
        # the norm, its sum with 1e-6, the factor and the product are rounded
        within(o, w, half(w, 5 * U * w.abs(), g.dtype) if g.dtype != F32 else 5 * U * w.abs() + TINY["f32"])
    if by == 1.0:
        assert all(torch.equal(g, o) for g, o in zip(grads, out))


def test_clip_odd_addresses_and_orders():
    """Views that start one element in, transposed and sliced: elements around them stay as they were."""
    flat = rand(1, 40001, dtype=BF)
    keep = flat.clone()
    grads = [flat[1:9000], flat[9001:19001].reshape(100, 100).t(), flat[20000:20001]]
    want = norm64(grads)
    n = tg.clip_grads(grads, 0.5)
    assert abs(float(n) - want) <= 2 * U * want
    for at in (0, 9000, 19001, 20001):
        assert flat[at] == keep[at]
    by = 0.5 / (want + 1e-6)
    w = keep[9001:19001].double() * by
    within(flat[9001:19001], w, half(w, 5 * U * w.abs(), BF))


def test_norm_range():
    """Squares beyond fp32's range, and gradients that are not finite."""
    for v in (1e30, 1e-30):
        g = [torch.full((5000,), v, device=DEV)]
        assert abs(float(tg.grad_norm(g)) / (v * math.sqrt(5000)) - 1) < 4 * U
    g = [torch.ones(10, device=DEV), torch.ones(9000, device=DEV)]
    g[1][8500] = float("nan")
    assert math.isnan(float(tg.clip_grads(g, 1.0))) and bool(g[0].isnan().all())
    g = [torch.ones(10, device=DEV), torch.ones(9000, device=DEV)]
    g[1][8500] = float("inf")
    assert math.isinf(float(tg.clip_grads(g, 1.0))) and bool((g[0] == 0).all()) and bool(g[1][8500].isnan())


def test_clip_with_a_given_norm():
    grads = some_grads(3, [1000, 70000])
    copies = [g.clone() for g in grads]
    n = tg.grad_norm(grads)
    two = (2 * n).clone()
    assert tg.clip_grads(grads, 1.0, given=two) is two
    by = torch.clamp(1.0 / (two + 1e-6), max=1.0)
    assert all(torch.equal(g, (c.float() * by).to(c.dtype)) for g, c in zip(grads, copies))


def test_norm_does_not_depend_on_addresses():
    grads = some_grads(5, [70000, 33, 8192 * 5 + 1])
    again = [torch.cat([g.new_zeros(3), g])[3:] for g in grads]
    assert torch.equal(tg.grad_norm(grads), tg.grad_norm(again))


# ---- grids of 256 x 256 tiles -------------------------------------------------------

# just over half the GPU's workgroups, one round and a ragged second, three rounds; one K tile, an odd and an even number
BIG = [(2048, 2040, 64), (2050, 2049, 200), (4100, 2300, 72), (4352, 2176, 328), (8000, 3400, 48)]


@pytest.mark.parametrize("m,f,k", BIG)
@pytest.mark.parametrize("dtype", [BF, FP], ids=KIND.get)
def test_glu_large_grids(m, f, k, dtype):
    x, wg, wu = rand(1, m, k, dtype=dtype), rand(2, f, k, dtype=dtype, scale=k ** -0.5), rand(3, f, k, dtype=dtype, scale=k ** -0.5)
    check_glu(x, wg, wu, "silu")
    out = [padded(torch.zeros(m, f, dtype=dtype, device=DEV), f + 1 + i, 7.0) for i in range(3)]
    check_glu(x, wg, wu, "relu", H=out[0], G=out[1], U=out[2])
    for o in out:
        whole = o.as_strided((m + 1, o.stride(0)), (o.stride(0), 1))
        assert bool((whole[:, f:] == 7).all()) and bool((whole[m] == 7).all())


@pytest.mark.parametrize("m,n,k", [(2048, 4090, 128), (2050, 4098, 400), (4100, 4700, 144), (8000, 7000, 96)])
@pytest.mark.parametrize("out", [F32, BF, FP], ids=KIND.get)
def test_int8_large_grids(m, n, k, out):
    check_int8(m, n, k, out)
    check_int8(m, n, k, out, "matrix", pads=(16, 32, 3))


@pytest.mark.parametrize("m,f,k", [(4000, 300, 3000), (600, 2100, 2100), (257, 4100, 2049)])
@pytest.mark.parametrize("dtype,grad", [(BF, BF), (BF, F32), (FP, FP)])
def test_glu_backward_large_grids(m, f, k, dtype, grad):
    check_backward(m, f, k, dtype, grad=grad, acc=True)


# ---- every tile size --------------------------------------------------------------

# (rows, columns) that reach each kernel by the count of tiles: few rows, 32 x 32 / 32 x 64, 64 x 64 in one and two
# groups, 64 x 128, 128 x 128 in two and one, at even sizes and at odd ones
TILES = [(9, 13000), (24, 9000), (33, 100), (70, 2000), (100, 4100), (64, 9000), (250, 4000), (500, 4030), (900, 4090), (1100, 6000)]


@pytest.mark.parametrize("m,n", TILES)
@pytest.mark.parametrize("k", [384, 1040, 203])
def test_int8_tiles(m, n, k):
    check_int8(m, n, k, BF)
    check_int8(m, n, k, F32, "matrix", pads=(16 - k % 16, 16 - k % 16, 0))


@pytest.mark.parametrize("m,f", [(m, n // 2) for m, n in TILES])
@pytest.mark.parametrize("k", [72, 520, 203])
def test_glu_tiles(m, f, k):
    x, wg, wu = rand(1, m, k), rand(2, f, k, scale=k ** -0.5), rand(3, f, k, scale=k ** -0.5)
    check_glu(x, wg, wu, "silu")


@pytest.mark.parametrize("m,k", [(33, 100), (70, 2000), (100, 4100), (250, 4000), (500, 4030), (900, 4090)])
def test_glu_backward_tiles(m, k):
    check_backward(m, 150, k, BF)


# both products of the backward pass in one launch of 256 x 256 tiles: evenly divided, one of them with fewer tiles than
# workgroups, sums of very different lengths, and without one of the products
@pytest.mark.parametrize("m,f,k", [(2100, 2100, 2050), (2048, 1024, 2560), (300, 6000, 2300), (6000, 200, 3100), (4200, 1000, 1500)])
@pytest.mark.parametrize("dtype,grad", [(BF, BF), (FP, F32)])
def test_glu_backward_one_launch(m, f, k, dtype, grad):
    check_backward(m, f, k, dtype, grad=grad, acc=True)


def test_glu_backward_parts_of_large_grids():
    """Each gradient alone is the same as both, up to the order of its sums."""
    m, f, k = 2100, 2100, 2050
    a = [rand(i, m, f) for i in range(3)] + [rand(3, m, k), rand(4, f, k, scale=0.05), rand(5, f, k, scale=0.05)]
    both = tg.gemm_glu_backward(*a, grad_dtype=F32)
    want, bound = ref.glu_backward(*a, "silu")
    dx, _, _ = tg.gemm_glu_backward(*a, weight_grad=False)
    _, dwg, dwu = tg.gemm_glu_backward(*a, input_grad=False, grad_dtype=F32)
    for got, w, b in zip((dx, dwg, dwu), want, bound):
        within(got, w, half(w, b, got.dtype))
    assert torch.equal(both[0], tg.gemm_glu_backward(*a, grad_dtype=F32)[0])


# ---- copies of unaligned operands -----------------------------------------------------

@pytest.mark.parametrize("m,n,k", [(2900, 3000, 77), (3000, 2900, 130), (2560, 4000, 1)])
def test_unaligned_large_grids(m, n, k):
    """Rows off 16 bytes in large grids: copied first, and without a workspace."""
    x, wg, wu = rand(1, m, k), rand(2, n // 2, k, scale=k ** -0.5), rand(3, n // 2, k, scale=k ** -0.5)
    assert tg.gemm_glu_workspace_bytes(m, n // 2, k) > 0 and tg.gemm_int8_workspace_bytes(m, n, k) > 0
    tiny = torch.empty(256, dtype=torch.uint8, device=DEV)
    check_glu(x, wg, wu, "silu")
    check_glu(x, wg, wu, "silu", workspace=tiny)
    check_glu(padded(x, k + 3), padded(wg, k + 8), wu, "silu")
    shifted = rand(1, m * 80 + 1)[1:].reshape(m, 80)
    check_glu(shifted, *(rand(i, n // 2, 80, scale=0.1) for i in (2, 3)), "gelu")
    check_int8(m, n, k, BF)
    check_int8(m, n, k, F32, "row", pads=(3, 16, 1))
    need = tg.gemm_glu_workspace_bytes(m, n // 2, k)
    guard = torch.full((need + 256,), 171, dtype=torch.uint8, device=DEV)
    assert torch.equal(tg.gemm_glu(x, wg, wu, workspace=guard[:need]), tg.gemm_glu(x, wg, wu)) and bool((guard[need:] == 171).all())
    with pytest.raises(tg.GemmError):
        tg.gemm_glu(x, wg, wu, workspace=guard[1:])


@pytest.mark.parametrize("m", [3, 150])
def test_matrices_next_to_each_other_in_one(m):
    """Operands as columns of one tensor, results as those of another: none is another's, and what lies behind them
    stays."""
    f, k = 96, 64
    ins, outs = torch.zeros(m, k + f, dtype=BF, device=DEV), torch.full((m, 3 * f + 8), 7.0, dtype=BF, device=DEV)
    x, dh, h, g, u = ins[:, :k], ins[:, k:], outs[:, :f], outs[:, f:2 * f], outs[:, 2 * f:3 * f]
    x.copy_(rand(1, m, k))
    dh.copy_(rand(2, m, f))
    w = rand(3, f, 2 * k)
    wg, wu = w[:, :k], w[:, k:]
    check_glu(x, wg, wu, "silu", H=h, G=g, U=u)
    dw = torch.full((f, 2 * k + 8), 7.0, device=DEV)
    dx, _, _ = tg.gemm_glu_backward(dh, g, u, x, wg, wu, dWg=dw[:, :k], dWu=dw[:, k:2 * k])
    alone = tg.gemm_glu_backward(dh.clone(), g.clone(), u.clone(), x.clone(), wg.clone(), wu.clone(), grad_dtype=F32)
    for got, want in zip((dx, dw[:, :k], dw[:, k:2 * k]), alone):
        assert torch.equal(got, want)
    tg.gemm_glu_backward(dh, g, u, x, wg, wu, Cg=dw[:, :k], Cu=dw[:, k:2 * k], dWg=dw[:, :k], dWu=dw[:, k:2 * k])
    for got, want in zip((dw[:, :k], dw[:, k:2 * k]), alone[1:]):
        # (one sum taken twice: exact)
        assert torch.equal(got, 2 * want)
    assert (outs[:, 3 * f:] == 7).all() and (dw[:, 2 * k:] == 7).all()


def test_clip_into_other_tensors_in_any_order():
    """Many tensors, results in another order in memory, some in place."""
    n = 600
    src = torch.randn(n, 40, device=DEV)
    dst = torch.zeros(n, 40, device=DEV)
    grads = [src[(7 * i) % n, :1 + i % 40] for i in range(n)]
    want, total = [g.clone() for g in grads], math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    out = [g if i % 3 == 0 else dst[(11 * i) % n, :1 + i % 40] for i, g in enumerate(grads)]
    norm = tg.clip_grads(grads, 1.0, out=out)
    assert abs(float(norm) - total) <= 2 * U * total
    for got, w in zip(out, want):
        # the factor's two roundings and the norm's, the product's
        within(got, w.double() / (total + 1e-6), 5 * U * w.double().abs() / total)


# ---- 256 x 128 tiles -------------------------------------------------------------------

# 235, 256 and 130 tiles, K of 8 to 33 tiles that ends inside one, results in whole pieces and not
@pytest.mark.parametrize("m,n", [(1100, 6000), (2048, 4096), (300, 8300), (1100, 5999)])
@pytest.mark.parametrize("k", [912, 1040, 2944, 4160])
def test_int8_narrow_tiles(m, n, k):
    for out in (BF, F32):
        check_int8(m, n, k, out)
        check_int8(m, n, k, out, "matrix", pads=(16, 32, 0))
    check_int8(m, n, k, FP, "matrix", pads=(0, 0, 3))
    check_int8(m, n, k, BF, "row")


@pytest.mark.parametrize("m,f,k", [(1100, 3000, 520), (2048, 2048, 464), (300, 4150, 1480), (1100, 2999, 1608)])
@pytest.mark.parametrize("dtype", [BF, FP], ids=KIND.get)
def test_glu_narrow_tiles(m, f, k, dtype):
    x, wg, wu = rand(1, m, k, dtype=dtype), rand(2, f, k, dtype=dtype, scale=k ** -0.5), rand(3, f, k, dtype=dtype, scale=k ** -0.5)
    check_glu(x, wg, wu, "gelu")
    out = [padded(torch.zeros(m, f, dtype=dtype, device=DEV), f + 8 + i, 7.0) for i in range(3)]
    check_glu(x, wg, wu, "silu", H=out[0], G=out[1], U=out[2])
    for o in out:
        whole = o.as_strided((m + 1, o.stride(0)), (o.stride(0), 1))
        assert bool((whole[:, f:] == 7).all()) and bool((whole[m] == 7).all())


@pytest.mark.parametrize("m,f,k", [(1000, 2728, 1024), (1001, 2731, 1003), (1600, 2731, 1003), (1100, 300, 6000)])
@pytest.mark.parametrize("dtype,grad", [(BF, BF), (BF, F32), (FP, FP)])
def test_glu_backward_narrow_tiles(m, f, k, dtype, grad):
    check_backward(m, f, k, dtype, grad=grad)
    check_backward(m, f, k, dtype, grad=grad, acc=True)


# ---- 128 x 128 tiles, one a CU ------------------------------------------------------

# 256 and 252 tiles; 1 to 5 K tiles and 17, which is once around the slots and more
@pytest.mark.parametrize("m,n", [(900, 4096), (500, 8000), (897, 4095)])
@pytest.mark.parametrize("k", [16, 144, 272, 400, 528, 2064])
def test_int8_single_tiles(m, n, k):
    check_int8(m, n, k, BF)
    check_int8(m, n, k, F32, "matrix", pads=(16, 32, 0))
    check_int8(m, n, k, FP, "matrix", pads=(0, 0, 3))


@pytest.mark.parametrize("m,f,k", [(1000, 2048, 64), (500, 4000, 136), (897, 2047, 200), (128, 14336, 264), (1000, 2048, 1040)])
@pytest.mark.parametrize("dtype", [BF, FP], ids=KIND.get)
def test_glu_single_tiles(m, f, k, dtype):
    x, wg, wu = rand(1, m, k, dtype=dtype), rand(2, f, k, dtype=dtype, scale=k ** -0.5), rand(3, f, k, dtype=dtype, scale=k ** -0.5)
    check_glu(x, wg, wu, "gelu_tanh")


@pytest.mark.parametrize("k", [1280, 1424])
def test_int8_narrow_tiles_of_other_counts(k):
    check_int8(2048, 4096, k, BF, "matrix")
    check_int8(1100, 6000, k, F32)


# ---- both products of a small backward pass in one launch -----------------------------

# up to 256 tiles of 64 x 64 and up to 1024, the longest sums and one K tile more, each gradient by itself
@pytest.mark.parametrize("m,f,k", [(64, 64, 64), (1, 30, 500), (355, 256, 1520), (179, 768, 1768), (200, 1024, 500), (200, 1025, 500),
                                   (2048, 64, 300), (2049, 64, 300), (500, 500, 500)])
@pytest.mark.parametrize("dtype,grad", [(BF, F32), (FP, FP)])
def test_glu_backward_small(m, f, k, dtype, grad):
    check_backward(m, f, k, dtype, grad=grad)
    check_backward(m, f, k, dtype, grad=grad, acc=True, name="gelu")
    a = [rand(i, m, f, dtype=dtype) for i in range(3)] + [rand(3, m, k, dtype=dtype), rand(4, f, k, dtype=dtype, scale=0.05),
                                                          rand(5, f, k, dtype=dtype, scale=0.05)]
    want, bound = ref.glu_backward(*a, "silu")
    dx, _, _ = tg.gemm_glu_backward(*a, weight_grad=False)
    _, dwg, dwu = tg.gemm_glu_backward(*a, input_grad=False, grad_dtype=grad)
    for got, w, b in zip((dx, dwg, dwu), want, bound):
        within(got, w, half(w, b, got.dtype))
