"""Row operators on the GPU against their 64-bit definitions: mxfp8_quantize
(every code and scale equal), rmsnorm, rmsnorm_mxfp8 and rmsnorm_backward
(within bounds derived from the roundings: tests/opsref.py), over all row
types, single elements to rows past the register kernels, strides, rows that
start at any element, in-place calls, and rows of zeros, infinities and NaN."""
import numpy as np
import pytest
import torch

import opsref as ref
import tiled_dense_gemm_tile_amd as tg

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
EPS = 1e-5


def f64(t):
    return t.detach().double().cpu().numpy()


def u8(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def rows_of(seed, rows, n, kind, pad=0, off=0, scale=1.0):
    """A (rows, n) device tensor of the type, `pad` elements between rows and
    the first element `off` elements into its storage, with a few large
    columns; the storage is returned with it."""
    rng = np.random.default_rng(seed)
    ld = n + pad
    store = rng.standard_normal(off + rows * ld + 8) * scale
    store[::37] *= 20
    s = torch.from_numpy(store.astype(np.float32)).to(DEV).to(TYPES[kind])
    return s[off:off + rows * ld].view(rows, ld)[:, :n]


QUANT = [(1, 32, 0, 0), (3, 64, 0, 0), (7, 96, 5, 3), (257, 160, 0, 1), (33, 4096, 32, 0), (5, 14336, 0, 0),
         (1000, 32, 1, 0)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("case", QUANT, ids=str)
def test_quantize(case, kind):
    rows, n, pad, off = case
    x = rows_of(1, rows, n, kind, pad, off)
    x[0, :32] = 0                                      # a block of zeros
    if rows > 2:
        x[2] *= 2.0 ** -13
    q, sf = tg.mxfp8_quantize(x)
    want, code = ref.quantize(f64(x))
    assert np.array_equal(u8(sf), code)
    assert np.array_equal(ref.e4m3(u8(q)), want)


def test_quantize_borders():
    """Block maxima at 448 * 2^e and one step to either side; elements halfway
    between codes; the smallest and largest numbers."""
    top = np.array([448.0, np.nextafter(np.float32(448), np.float32(0)), np.nextafter(np.float32(448), np.float32(1e9)),
                    256.0, 1.0, 1.75, 1.7500001, 2.0 ** -118, 2.0 ** -126, 2.0 ** -149, 3.4e38, 2.0 ** 127], np.float32)
    x = np.zeros((top.size, 32), np.float32)
    x[:, 0] = top
    for i in range(1, 31):                             # ties between neighbouring codes, of every binade
        x[:, i] = -top / 2 ** (i % 20) * np.float32((17 + 2 * (i % 8)) / 32)
    q, sf = tg.mxfp8_quantize(torch.from_numpy(x).to(DEV))
    want, code = ref.quantize(x.astype(np.float64))
    assert np.array_equal(u8(sf), code)
    assert np.array_equal(ref.e4m3(u8(q)), want)
    assert np.nanmax(np.abs(want)) <= 448


@pytest.mark.parametrize("kind", TYPES)
def test_quantize_nonfinite(kind):
    x = rows_of(2, 6, 96, kind)
    x[0, 5], x[1, 40], x[2, 70] = float("nan"), float("inf"), float("-inf")
    x[3, 32:64] = float("nan")
    q, sf = tg.mxfp8_quantize(x)
    want, code = ref.quantize(f64(x))
    assert np.array_equal(u8(sf), code)
    assert np.array_equal(ref.e4m3(u8(q)), want, equal_nan=True)
    assert np.isnan(want).sum() == 35


def test_quantize_leaves_padding():
    x = rows_of(3, 40, 64, "bf16")
    qs = torch.full((41, 80), 0x5A, dtype=torch.uint8, device=DEV)
    ss = torch.full((41, 5), 0x5A, dtype=torch.uint8, device=DEV)
    tg.mxfp8_quantize(x, Q=qs[:40, 3:67], SF=ss[:40, 1:3])
    want, code = ref.quantize(f64(x))
    q, s = u8(qs), u8(ss)
    assert np.array_equal(ref.e4m3(q[:40, 3:67]), want) and np.array_equal(s[:40, 1:3], code)
    q[:40, 3:67], s[:40, 1:3] = 0x5A, 0x5A
    assert (q == 0x5A).all() and (s == 0x5A).all()


def test_quantize_empty():
    for shape in ((0, 64), (5, 0)):
        q, sf = tg.mxfp8_quantize(torch.zeros(shape, dtype=torch.bfloat16, device=DEV))
        assert q.shape == shape and sf.shape == (shape[0], shape[1] // 32)


# (rows, n, pad, offset): a wave per row, a workgroup per row, the long kernel
NORM = [(1, 1, 0, 0), (3, 7, 2, 1), (5, 32, 0, 0), (2, 257, 0, 3), (9, 1000, 0, 0), (1, 4096, 0, 0), (1030, 96, 0, 1),
        (1027, 4096, 8, 0), (1025, 1001, 0, 0), (4, 8193, 1, 0), (3, 14336, 0, 5), (2, 16384, 0, 0), (2, 32768, 0, 0),
        (2, 40001, 0, 1)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("case", NORM, ids=str)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(case, kind, residual):
    rows, n, pad, off = case
    x = rows_of(4, rows, n, kind, pad, off)
    r = rows_of(5, rows, n, kind, 0, off) if residual else None
    w = rows_of(6, 1, n, kind if n % 3 else "f32")[0].contiguous()
    y, h, rstd = tg.rmsnorm(x, w, EPS, residual=r)
    hv = f64(h)
    if residual:
        # the sum is formed in fp32 and rounded again: half a step, and fp32's
        s = f64(x) + f64(r)
        assert (np.abs(hv - s) <= (ref.HALF[kind] + (ref.U if kind != "f32" else 0)) * np.abs(s) + ref.TINY[kind]).all()
    else:
        assert h is x
    want, rs = ref.norm(hv, f64(w), EPS)
    assert (np.abs(f64(rstd) - rs) <= ref.rstd_bound(n) * rs).all()
    # (h w) rstd: two roundings beside rstd's error, then the output's
    bound = (ref.rstd_bound(n) + 2 * ref.U) * np.abs(want) + 2.0 ** -148
    assert (np.abs(f64(y) - want) <= bound + ref.HALF[kind] * (np.abs(want) + bound) + ref.TINY[kind]).all()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("case", [(1, 32, 0, 0), (3, 96, 1, 1), (7, 1024, 0, 0), (1025, 416, 0, 3), (1026, 4096, 0, 0),
                                  (2, 8224, 0, 0), (3, 16384, 32, 0), (2, 40032, 0, 1)], ids=str)
def test_norm_mxfp8(case, kind):
    rows, n, pad, off = case
    x, r = rows_of(7, rows, n, kind, pad, off), rows_of(8, rows, n, kind)
    w = rows_of(9, 1, n, kind)[0].contiguous()
    q, sf, h, rstd = tg.rmsnorm_mxfp8(x, w, EPS, residual=r)
    y16, h16, rstd16 = tg.rmsnorm(x, w, EPS, residual=r)
    assert torch.equal(h, h16) and torch.equal(rstd, rstd16)
    want, rs = ref.norm(f64(h), f64(w), EPS)
    assert (np.abs(f64(rstd) - rs) <= ref.rstd_bound(n) * rs).all()
    d = (ref.rstd_bound(n) + 2 * ref.U) * np.abs(want)
    e = u8(sf).astype(np.int64) - 127
    amax, slack = np.abs(want).reshape(rows, -1, 32).max(axis=2), d.reshape(rows, -1, 32).max(axis=2)
    # the least scale that clips nothing, of a maximum known to within `slack`
    assert (amax - slack <= 448 * np.ldexp(1.0, e)).all()
    assert ((amax + slack > 448 * np.ldexp(1.0, e - 1)) | (e == -127)).all()
    # half a step of e4m3: 2^-4 of the value, or 2^-10 of the scale below its normal range
    step = np.maximum(2.0 ** -4 * (np.abs(want) + d), np.repeat(np.ldexp(1.0, e - 10), 32, axis=1))
    assert (np.abs(ref.dequant(u8(q), u8(sf)) - want) <= step + d).all()


@pytest.mark.parametrize("where", ["x", "r", "y_over_x", "y_over_r"])
@pytest.mark.parametrize("n", [96, 8192, 40000])
def test_norm_in_place(where, n):
    x, r = rows_of(10, 5, n, "bf16"), rows_of(11, 5, n, "bf16")
    w = rows_of(12, 1, n, "bf16")[0].contiguous()
    y0, h0, s0 = tg.rmsnorm(x, w, EPS, residual=r)
    a, b = x.clone(), r.clone()
    kw = {"x": dict(H=a), "r": dict(H=b), "y_over_x": dict(Y=a), "y_over_r": dict(Y=b)}[where]
    y, h, s = tg.rmsnorm(a, w, EPS, residual=b, **kw)
    assert torch.equal(y, y0) and torch.equal(h, h0) and torch.equal(s, s0)
    assert (h if "H" in kw else y).data_ptr() == next(iter(kw.values())).data_ptr()


def test_norm_special_rows():
    x = rows_of(13, 6, 256, "f32")
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 9] = float("inf")
    w = torch.ones(256, device=DEV)
    y, _, rstd = tg.rmsnorm(x, w, EPS)
    assert (y[0] == 0).all() and abs(rstd[0].item() - EPS ** -0.5) < 1e-4 * EPS ** -0.5
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 9])
    want, _ = ref.norm(f64(x[3:]), np.ones(256), EPS)
    assert np.abs(f64(y[3:]) - want).max() < 1e-5      # the other rows do not notice
    q, sf, _, _ = tg.rmsnorm_mxfp8(x, w, EPS)
    v = ref.e4m3(u8(q))
    assert (v[0] == 0).all() and (u8(sf)[0] == 0).all()
    assert np.isnan(v[1]).all() and np.isnan(v[2, 9]) and np.isfinite(v[3:]).all()


def test_norm_leaves_padding():
    x = rows_of(14, 9, 100, "bf16")
    w = torch.ones(100, dtype=torch.bfloat16, device=DEV)
    big = torch.full((10, 111), 3.5, dtype=torch.bfloat16, device=DEV)
    hs = torch.full((10, 107), 4.5, dtype=torch.bfloat16, device=DEV)
    y0, h0, _ = tg.rmsnorm(x, w, EPS, residual=x)
    tg.rmsnorm(x, w, EPS, residual=x, Y=big[:9, 5:105], H=hs[:9, 1:101])
    assert torch.equal(big[:9, 5:105], y0) and torch.equal(hs[:9, 1:101], h0)
    big[:9, 5:105], hs[:9, 1:101] = 3.5, 4.5
    assert (big == 3.5).all() and (hs == 4.5).all()


BWD = [(1, 1, 0, 0), (3, 7, 2, 1), (5, 1000, 0, 0), (1500, 100, 0, 1), (2049, 2048, 0, 0), (1100, 4100, 4, 0),
       (40, 8192, 0, 0), (9, 14336, 0, 3), (5, 16384, 0, 0), (70, 20001, 0, 1)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("case", BWD, ids=str)
@pytest.mark.parametrize("extra", [False, True])
def test_norm_backward(case, kind, extra):
    rows, n, pad, off = case
    h, dy = rows_of(20, rows, n, kind, pad, off), rows_of(21, rows, n, kind, 0, off, 0.1)
    dh = rows_of(22, rows, n, kind, 3, 0, 0.1) if extra else None
    w = rows_of(23, 1, n, kind if n % 3 else "f32")[0].contiguous()
    rstd = torch.from_numpy((1 / np.sqrt((f64(h) ** 2).mean(1) + EPS)).astype(np.float32)).to(DEV)
    dx, dw = tg.rmsnorm_backward(dy, h, w, rstd, dH=dh)
    want, wdw, ag, au, adw = ref.norm_backward(f64(dy), f64(h), f64(w), f64(rstd), 0.0 if dh is None else f64(dh))
    # g: a rounding; u = h rstd: one; the row's sum: its chain of n / 64 + 32,
    # its terms' three roundings, the mean's division; u m, g - u m, the last
    # product and sum: one each of at most their terms
    bound = 4 * ref.U * ag + (n / 64 + 32 + 9) * ref.U * au + 2 * ref.U * np.abs(want)
    assert (np.abs(f64(dx) - want) <= bound + ref.HALF[kind] * (np.abs(want) + bound) + ref.TINY[kind]).all()
    # a column's chain: a group's rows (at least 64 groups, or a group a row),
    # 32 partial sums a lane and 32 lanes; two roundings a term
    assert (np.abs(f64(dw) - wdw) <= (rows / 64 + 1 + 64 + 2) * ref.U * adw).all()
    dx2, none = tg.rmsnorm_backward(dy, h, w, rstd, dH=dh, weight_grad=False)
    assert none is None and torch.equal(dx, dx2)


@pytest.mark.parametrize("n", [96, 8192, 20000])
def test_norm_backward_in_place(n):
    h, dy, dh = (rows_of(s, 70, n, "bf16") for s in (24, 25, 26))
    w = rows_of(27, 1, n, "bf16")[0].contiguous()
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    dx0, dw0 = tg.rmsnorm_backward(dy, h, w, rstd, dH=dh)
    for over in ("dy", "dh"):
        a, b = dy.clone(), dh.clone()
        t = a if over == "dy" else b
        dx, dw = tg.rmsnorm_backward(a, h, w, rstd, dH=b, dX=t)
        assert dx.data_ptr() == t.data_ptr() and torch.equal(dx, dx0) and torch.equal(dw, dw0)


def test_norm_backward_no_rows():
    e = torch.zeros(0, 48, device=DEV)
    dx, dw = tg.rmsnorm_backward(e, e, torch.ones(48, device=DEV), torch.zeros(0, device=DEV),
                                 dW=torch.full((48,), 7.0, device=DEV))
    assert dx.shape == (0, 48) and (dw == 0).all()


def test_norm_backward_leaves_what_lies_behind():
    h = rows_of(28, 300, 100, "bf16")
    w = torch.ones(100, dtype=torch.bfloat16, device=DEV)
    rstd = torch.ones(300, device=DEV)
    need = tg.rmsnorm_backward_workspace_bytes(300, 100)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    dw, dx = torch.full((130,), 9.0, device=DEV), torch.full((301, 107), 4.5, dtype=torch.bfloat16, device=DEV)
    tg.rmsnorm_backward(h, h, w, rstd, dX=dx[:300, 2:102], dW=dw[:100], workspace=ws[:need])
    assert (ws[need:] == 0x5A).all() and (dw[100:] == 9).all()
    dx[:300, 2:102] = 4.5
    assert (dx == 4.5).all()


def test_norm_gradient_against_differences():
    """dx and dw along random directions against central differences of the
    64-bit forward form.  With steps of 1e-4 of unit-variance rows the
    difference's own error is of the order of 1e-8 of the loss's third
    derivative; fp32's is (n / 64 + 41) u of the sums' magnitudes, under
    1e-5 of |dy| |direction| here."""
    rng = np.random.default_rng(30)
    h, dy, w = rng.standard_normal((6, 640)), rng.standard_normal((6, 640)), 1 + 0.1 * rng.standard_normal(640)
    h, dy, w = (a.astype(np.float32).astype(np.float64) for a in (h, dy, w))
    d = [torch.from_numpy(a.astype(np.float32)).to(DEV) for a in (h, dy, w)]
    _, _, rstd = tg.rmsnorm(d[0], d[2], EPS)
    dx, dw = tg.rmsnorm_backward(d[1], d[0], d[2], rstd)
    for seed in range(4):
        r = np.random.default_rng(seed)
        vh, vw = r.standard_normal(h.shape), r.standard_normal(w.shape)
        for a, b, got in ((vh, 0 * vw, (f64(dx) * vh).sum()), (0 * vh, vw, (f64(dw) * vw).sum())):
            loss = lambda t: (ref.norm(h + t * a, w + t * b, EPS)[0] * dy).sum()  # noqa: E731
            num = (loss(1e-4) - loss(-1e-4)) / 2e-4
            assert abs(got - num) <= 1e-5 * np.linalg.norm(dy) * max(np.linalg.norm(a), np.linalg.norm(b) * np.sqrt(6))


def test_same_bits_every_call():
    h, dy = rows_of(31, 3000, 1000, "bf16"), rows_of(32, 3000, 1000, "bf16")
    w = rows_of(33, 1, 1000, "bf16")[0].contiguous()
    y, _, rstd = tg.rmsnorm(h, w, EPS)
    first = tg.rmsnorm_backward(dy, h, w, rstd)
    for _ in range(3):
        again = tg.rmsnorm_backward(dy, h, w, rstd)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        assert torch.equal(y, tg.rmsnorm(h, w, EPS)[0])


@pytest.mark.parametrize("case", [((4 << 20) + 7, 8, "bf16"), ((2 << 20) + 3, 260, "f32")], ids=str)
def test_norm_of_more_rows_than_one_launch(case):
    """2^20 workgroups of four or two rows each, and a few rows more."""
    rows, n, kind = case
    x = torch.randn(rows, n, device=DEV, generator=torch.Generator(DEV).manual_seed(40)).to(TYPES[kind])
    w = rows_of(41, 1, n, "f32")[0].contiguous()
    y, _, rstd = tg.rmsnorm(x, w, EPS, Y=torch.full_like(x, float("nan")), rstd=torch.full((rows,), -1.0, device=DEV))
    for a in (0, rows // 2, rows - 4099):
        want, rs = ref.norm(f64(x[a:a + 4099]), f64(w), EPS)
        assert (np.abs(f64(rstd[a:a + 4099]) - rs) <= ref.rstd_bound(n) * rs).all()
        bound = (ref.rstd_bound(n) + 2 * ref.U) * np.abs(want) + 2.0 ** -148
        assert (np.abs(f64(y[a:a + 4099]) - want) <= bound + ref.HALF[kind] * (np.abs(want) + bound) + ref.TINY[kind]).all()
    assert (rstd > 0).all() and not torch.isnan(y).any()


def test_long_rows_past_the_grid():
    """More rows than the kernels of long rows have workgroups: each as if alone."""
    rows, n = 2051, 16388
    x, dy = (torch.randn(rows, n, device=DEV, generator=torch.Generator(DEV).manual_seed(s)) for s in (42, 43))
    w = rows_of(44, 1, n, "f32")[0].contiguous()
    y, _, rstd = tg.rmsnorm(x, w, EPS)
    dx, dw = tg.rmsnorm_backward(dy, x, w, rstd)
    for a in (0, 1500, 2047):
        yb, _, rb = tg.rmsnorm(x[a:a + 4], w, EPS)
        assert torch.equal(y[a:a + 4], yb) and torch.equal(rstd[a:a + 4], rb)
        assert torch.equal(dx[a:a + 4], tg.rmsnorm_backward(dy[a:a + 4], x[a:a + 4], w, rb, weight_grad=False)[0])
    want, rs = ref.norm(f64(x[2040:]), f64(w), EPS)
    assert (np.abs(f64(rstd[2040:]) - rs) <= ref.rstd_bound(n) * rs).all()
    u = x.double() * rstd.double()[:, None]
    adw = (dy.double() * u).abs().sum(0)
    assert ((dw.double() - (dy.double() * u).sum(0)).abs() <= (rows / 64 + 1 + 64 + 2) * ref.U * adw).all()


@pytest.mark.parametrize("n", [32, 1024, 4096, 8192, 14336])
@pytest.mark.parametrize("residual", [False, True])
def test_a_row_does_not_depend_on_its_batch(n, residual):
    x, r = rows_of(48, 3000, n, "bf16"), rows_of(49, 3000, n, "bf16")
    w = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    y, h, rstd = tg.rmsnorm(x, w, EPS, residual=r if residual else None)
    for a, b in ((0, 1), (2999, 3000), (700, 733)):
        ya, ha, sa = tg.rmsnorm(x[a:b], w, EPS, residual=r[a:b] if residual else None)
        assert torch.equal(ya, y[a:b]) and torch.equal(ha, h[a:b]) and torch.equal(sa, rstd[a:b])


def test_norm_over_its_input_returns_no_h():
    x = rows_of(45, 5, 96, "bf16")
    w = rows_of(46, 1, 96, "bf16")[0].contiguous()
    y0, h, s0 = tg.rmsnorm(x, w, EPS)
    assert h is x
    a = x.clone()
    y, h, s = tg.rmsnorm(a, w, EPS, Y=a)
    assert h is None and torch.equal(y, y0) and torch.equal(s, s0) and y.data_ptr() == a.data_ptr()
    e = torch.zeros(0, 96, dtype=torch.bfloat16, device=DEV)
    assert tg.rmsnorm(e, w, EPS)[1] is e


def test_norm_of_infinite_rows():
    x = rows_of(47, 3, 256, "f32")
    x[0, 9] = float("inf")
    x[1] *= 1e20                                       # squares past fp32
    y, _, rstd = tg.rmsnorm(x, torch.ones(256, device=DEV), EPS)
    assert rstd[0] == 0 and rstd[1] == 0 and (y[1] == 0).all()
    assert torch.isnan(y[0, 9]) and (y[0, :9] == 0).all() and (y[0, 10:] == 0).all()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("base", [0, 504, 2040, 4096, 8192])
def test_every_row_end(kind, base):
    """Rows that end at every element of a vector, forward and backward, in surroundings that stay as they are."""
    w = rows_of(50, 1, base + 9, "f32")[0].contiguous()
    for n in range(base + 1, base + 9):
        x, r, dy = (rows_of(s, 5, n, kind, 3, 1) for s in (51, 52, 53))
        big = torch.full((7, n + 5), 7.0, dtype=TYPES[kind], device=DEV)
        y, h, rstd = tg.rmsnorm(x, w[:n], EPS, residual=r, Y=big[1:6, 2:n + 2])
        want, rs = ref.norm(f64(h), f64(w[:n]), EPS)
        s = f64(x) + f64(r)
        assert (np.abs(f64(h) - s) <= (ref.HALF[kind] + (ref.U if kind != "f32" else 0)) * np.abs(s) + ref.TINY[kind]).all()
        assert (np.abs(f64(rstd) - rs) <= ref.rstd_bound(n) * rs).all()
        bound = (ref.rstd_bound(n) + 2 * ref.U) * np.abs(want) + 2.0 ** -148
        assert (np.abs(f64(y) - want) <= bound + ref.HALF[kind] * (np.abs(want) + bound) + ref.TINY[kind]).all()
        big[1:6, 2:n + 2] = 7
        assert (big == 7).all()
        dx, dw = tg.rmsnorm_backward(dy, h, w[:n], rstd, dH=x, dX=big[1:6, 2:n + 2])
        want, wdw, ag, au, adw = ref.norm_backward(f64(dy), f64(h), f64(w[:n]), f64(rstd), f64(x))
        bound = 4 * ref.U * ag + (n / 64 + 32 + 9) * ref.U * au + 2 * ref.U * np.abs(want)
        assert (np.abs(f64(dx) - want) <= bound + ref.HALF[kind] * (np.abs(want) + bound) + ref.TINY[kind]).all()
        assert (np.abs(f64(dw) - wdw) <= (1 + 1 + 64 + 2) * ref.U * adw).all()
        big[1:6, 2:n + 2] = 7
        assert (big == 7).all()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("case", [(2048, 4096), (5000, 96), (3001, 512), (4097, 1024), (1500, 2304), (700, 8192),
                                  (500, 14336), (301, 40032)], ids=str)
def test_codes_of_the_norm_are_those_of_the_64_bit_result(kind, case):
    """rmsnorm_mxfp8 takes what fp32's roundings could change in 64 bits: codes and scales equal those of the 64-bit
    y, whose own error of 2^-45 lies a million times nearer to a border than any of these values.  The same bits
    every call."""
    rows, n = case
    x, r = rows_of(50, rows, n, kind), rows_of(51, rows, n, kind)
    w = rows_of(52, 1, n, kind if n % 3 else "f32")[0].contiguous()
    q, sf, h, rstd = tg.rmsnorm_mxfp8(x, w, EPS, residual=r)
    for _ in range(3):
        for a, b in zip((q, sf, h, rstd), tg.rmsnorm_mxfp8(x, w, EPS, residual=r)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    y, rs = ref.norm(f64(h), f64(w), EPS)
    want, code = ref.quantize(y)
    assert np.array_equal(u8(sf), code) and np.array_equal(ref.e4m3(u8(q)), want)
    assert (np.abs(f64(rstd) - rs) <= ref.U * rs).all()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("h", [1.0, 0.25])
def test_norm_codes_on_and_beside_the_borders(kind, h):
    """Rows of one magnitude and eps 0: y is +-w itself.  Weights in the middle of two neighbouring codes (to even),
    and one fp32 step to either side; block maxima at 448 steps of a scale and beside it."""
    codes = np.arange(0, 127)
    mid = (ref.e4m3(codes[:-1].astype(np.uint8)) + ref.e4m3(codes[1:].astype(np.uint8))) / 2
    rng = np.random.default_rng(53)
    rows = []
    for k in range(40):
        b = rng.permutation(mid)[:31 * 4].reshape(4, 31)
        b = np.concatenate((b, np.full((4, 1), 448.0)), axis=1)
        rows.append((b * 2.0 ** rng.integers(-30, 30)).reshape(-1))
    w = np.concatenate(rows).astype(np.float32)
    step = rng.integers(-1, 2, w.shape)
    w = np.where(step > 0, np.nextafter(w, np.float32(np.inf)), np.where(step < 0, np.nextafter(w, np.float32(0)), w))
    n = w.size
    sign = rng.choice([-1.0, 1.0], size=(3, n))
    x = torch.from_numpy(sign * h).to(DEV).to(TYPES[kind])
    q, sf, _, rstd = tg.rmsnorm_mxfp8(x, torch.from_numpy(w).to(DEV), 0.0)
    assert (rstd == 1 / h).all()
    want, code = ref.quantize(sign * w.astype(np.float64))
    assert np.array_equal(u8(sf), code) and np.array_equal(ref.e4m3(u8(q)), want)


def test_rows_without_a_norm():
    """eps 0: a row of zeros, one of small values; with any eps: one whose sum of squares is past fp32."""
    x = torch.zeros(4, 96, device=DEV)
    x[1, ::2] = -2.0 ** -100
    x[2], x[3] = 2.0 ** 80, 1.0
    w = torch.full((96,), 2.0, device=DEV)
    y, _, rstd = tg.rmsnorm(x, w, 0.0)
    assert torch.isinf(rstd[0]) and rstd[2] == 0 and rstd[3] == 1
    assert torch.isnan(y[0]).all() and (y[1, 1::2] == 0).all() and (y[2] == 0).all() and (y[3] == 2).all()
    assert (np.abs(f64(y[1, ::2]) + 8 ** 0.5) <= 3 * ref.U * 8 ** 0.5).all()
    q, sf, _, _ = tg.rmsnorm_mxfp8(x, w, 0.0)
    v = ref.dequant(u8(q), u8(sf))
    assert np.isnan(v[0]).all() and (v[2] == 0).all() and (v[3] == 2).all()
    assert (np.abs(v[1, ::2] + 8 ** 0.5) <= 2.0 ** -4 * 8 ** 0.5).all() and (v[1, 1::2] == 0).all()
    y, _, _ = tg.rmsnorm(x, w, EPS)
    assert (y[0] == 0).all() and (y[2] == 0).all() and torch.isfinite(y).all()


@pytest.mark.parametrize("kind", TYPES)
def test_norm_codes_beside_weights_that_are_not_finite(kind):
    """NaN codes at them, and block scales as if they were zero."""
    x = rows_of(54, 5, 256, kind)
    w = rows_of(55, 1, 256, "f32")[0].contiguous()
    w[3], w[40], w[200] = float("inf"), float("nan"), -float("inf")
    q, sf, h, _ = tg.rmsnorm_mxfp8(x, w, EPS)
    y, _ = ref.norm(f64(h), f64(w), EPS)
    want, code = ref.quantize(y)
    assert np.array_equal(u8(sf), code) and np.array_equal(ref.e4m3(u8(q)), want, equal_nan=True)
    assert np.isnan(want).sum() == 15
