"""Operands of the operators around the block-scaled products that reach past
4 GiB: rows far apart give the same bits as packed ones."""
import pytest
import torch

import tiled_dense_gemm_tile_amd as tg

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def far(t, ld):
    """t with `ld` elements between the starts of its rows."""
    rows, n = t.shape
    v = torch.empty(rows * ld, dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device=DEV)
    v = v.view(t.dtype).view(rows, ld)[:, :n]
    v.copy_(t)
    assert (rows - 1) * ld * t.element_size() > 1 << 32
    return v


def test_row_operators():
    rows, n, ld = 2200, 992, (1 << 20) + 8
    x, dy = (torch.randn(rows, n, device=DEV, generator=gen(s)).bfloat16() for s in (1, 2))
    w = torch.randn(n, device=DEV, generator=gen(3))
    y, _, rstd = tg.rmsnorm(x, w, 1e-5)
    xf = far(x, ld)
    assert torch.equal(tg.rmsnorm(xf, w, 1e-5, Y=far(torch.zeros_like(x), ld))[0], y)
    dx, dw = tg.rmsnorm_backward(dy, x, w, rstd)
    dxf, dwf = tg.rmsnorm_backward(far(dy, ld), xf, w, rstd, dX=xf.new_empty(rows * ld).view(rows, ld)[:, :n])
    assert torch.equal(dxf, dx) and torch.equal(dwf, dw)
    del dxf
    q, sf = tg.mxfp8_quantize(x)
    qf, sff = tg.mxfp8_quantize(xf, Q=far(torch.zeros(rows, n, dtype=torch.uint8, device=DEV), 2 * ld))
    assert torch.equal(qf, q.view(torch.uint8)) and torch.equal(sff.view(torch.uint8), sf.view(torch.uint8))


@pytest.mark.parametrize("off", [0, 1])
def test_weight_gradient(off):
    """Rows on 16 bytes and one element off (the kernel that takes every call)."""
    m, n, k = 1100, 320, 1100
    a = torch.randn(k, m, device=DEV, generator=gen(4)).bfloat16()
    q, sf = tg.mxfp8_quantize(torch.randn(k, n, device=DEV, generator=gen(5)).bfloat16())
    q = q.view(torch.uint8)
    lda, ldb = (1 << 21) - 8 + off, (1 << 22) - 16 + off
    af, qf = far(a, lda), far(q, ldb)
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    pad = 8 + off                                       # rows as far off 16 bytes, near each other
    an = torch.empty(k, m - m % 8 + 8 + pad, dtype=a.dtype, device=DEV)[:, :m].copy_(a)
    qn = torch.empty(k, n + 16 + off, dtype=q.dtype, device=DEV)[:, :n].copy_(q)
    want = tg.gemm_wgrad_mxfp8(an, qn, sf, workspace=none)
    D = tg.gemm_wgrad_mxfp8(af, qf, sf, D=far(torch.zeros(m, n, device=DEV), (1 << 20) + 4), workspace=none)
    assert torch.equal(D, want)
    v = torch.ldexp(q.view(torch.float8_e4m3fn).double().view(k, n // 32, 32),
                    sf.view(torch.uint8).int()[:, :, None] - 127).view(k, n)
    exact, size = (torch.mm(s.t().contiguous(), t) for s, t in ((a.double(), v), (a.double().abs(), v.abs())))
    assert ((want.double() - exact).abs() <= k * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("off", [0, 1])
def test_gemv(off):
    m, n, k = 5, 1100, 2048
    x = torch.randn(m, k, device=DEV, generator=gen(6)).bfloat16()
    w = torch.randint(0, 256, (n, k // 2), device=DEV, generator=gen(7), dtype=torch.uint8)
    sf = torch.randint(116, 122, (n, k // 32), device=DEV, generator=gen(8), dtype=torch.uint8)
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    near = torch.empty(n, k // 2 + 16 + off, dtype=torch.uint8, device=DEV)[:, :k // 2].copy_(w)
    want = tg.gemv_mxfp4(x, near, sf, workspace=none)
    assert torch.equal(tg.gemv_mxfp4(x, far(w, (1 << 22) - 16 + off), sf, workspace=none), want)
    # the same sums in another order: k half steps of their magnitudes each
    size = tg.gemv_mxfp4(x.abs(), w & 0x77, sf)
    assert ((want - tg.gemv_mxfp4(x, w, sf)).abs() <= 2 * (k + 1) * 2.0 ** -24 * size).all()
