"""The feed-forward layer's operators on operands past 2^31 elements and 4
GiB: first, last and sampled results against the definition in 64 bits."""
import math

import pytest
import torch

import layersref as ref
import tiled_dense_gemm_tile_amd as tg
from layersref import DEV, U, half, rand, within

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def some(n, seed=0):
    """First, last and sampled indexes of n."""
    g = torch.Generator().manual_seed(seed)
    return torch.cat([torch.tensor([0, n - 1, n // 2]), torch.randint(0, n, (61,), generator=g)]).to(DEV)


def test_glu_results():
    m, f, k = 160000, 14400, 16
    x, wg, wu = rand(1, m, k), rand(2, f, k), rand(3, f, k)
    h, g, u = tg.gemm_glu(x, wg, wu, keep=True)
    i, j = some(m), some(f, 1)
    want, bound = ref.glu(x[i], wg[j], wu[j], "silu")
    for got, w, b in zip((h, g, u), want, bound):
        within(got[i][:, j], w, half(w, b, BF))


@pytest.mark.parametrize("m", [2, 40])
def test_int8_weights(m):
    n, k = 520000, 8320
    a = torch.randint(-127, 128, (m, k), device=DEV, dtype=torch.int8)
    b = torch.randint(-127, 128, (n, k), device=DEV, dtype=torch.int8)
    sa, sb = torch.rand(m, device=DEV), torch.rand(n, device=DEV)
    d = tg.gemm_int8(a, sa, b, sb)
    j = some(n)
    want = (a.double() @ b[j].double().t()) * sa.double()[:, None] * sb[j].double()
    within(d[:, j], want, 3 * U * want.abs())


def test_int8_rows():
    m, n, k = 600000, 4096, 4096
    a = torch.randint(-127, 128, (m, k), device=DEV, dtype=torch.int8)
    b = torch.randint(-127, 128, (n, k), device=DEV, dtype=torch.int8)
    sa, sb = torch.rand(m, device=DEV), torch.rand(n, device=DEV)
    d = tg.gemm_int8(a, sa, b, sb, out_dtype=BF)
    i = some(m)
    want = (a[i].double() @ b.double().t()) * sa[i].double()[:, None] * sb.double()
    within(d[i], want, half(want, 3 * U * want.abs(), BF))


def test_quantize():
    rows, n = 140000, 16400
    x = torch.empty(rows, n, dtype=BF, device=DEV)
    for lo in range(0, rows, 20000):
        x[lo:lo + 20000] = rand(lo, min(20000, rows - lo), n)
    q, s = tg.int8_quantize(x)
    i = some(rows)
    wq, ws = ref.quantize(x[i])
    assert torch.equal(q[i], wq) and torch.equal(s[i], ws)


def test_glu_backward():
    m, f, k = 40000, 30000, 48
    dh, g, u = (rand(i, m, f) for i in range(3))
    x, wg, wu = rand(3, m, k), rand(4, f, k), rand(5, f, k)
    dx, dwg, dwu = tg.gemm_glu_backward(dh, g, u, x, wg, wu, grad_dtype=F32)
    i, j = some(m), some(f, 1)
    want, bound = ref.glu_backward(dh[i], g[i], u[i], x[i], wg, wu, "silu")
    within(dx[i], want[0], half(want[0], bound[0], BF))
    want, bound = ref.glu_backward(dh[:, j].contiguous(), g[:, j].contiguous(), u[:, j].contiguous(), x, wg[j], wu[j], "silu")
    within(dwg[j], want[1], half(want[1], bound[1], F32))
    within(dwu[j], want[2], half(want[2], bound[2], F32))


def test_clip():
    n = (1 << 31) + 12345
    g = torch.full((n,), 0.5, dtype=BF, device=DEV)
    g[-1] = 3.0
    want = math.sqrt(0.25 * (n - 1) + 9.0)
    assert abs(float(tg.clip_grads([g, torch.ones(3, device=DEV)], 1.0)) - math.sqrt(want ** 2 + 3)) <= 2 * U * want
    by = 1.0 / (math.sqrt(want ** 2 + 3) + 1e-6)
    for at, v in ((0, 0.5), (n // 2, 0.5), (n - 2, 0.5), (n - 1, 3.0)):
        assert abs(float(g[at]) - v * by) <= (2.0 ** -8 + 5 * U) * v * by
