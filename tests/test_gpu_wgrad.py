"""gemm_wgrad_mxfp8 on the GPU: exact on integer values (every product and
partial sum an integer below 2^24), within |D - D_ref| <= K 2^-24 sum|a b| on
random ones, over single tokens to long sums, ragged sizes, rows that start
at any element, strides, C and in-place accumulation, cut and uncut K."""
import numpy as np
import pytest
import torch

import opsref as ref
import tiled_dense_gemm_tile_amd as tg

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
OUT = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().double().cpu().numpy()


def u8(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def strided(a, dtype, pad, off):
    """The host matrix as a device tensor with `pad` elements between rows, `off` before the first."""
    rows, n = a.shape
    s = torch.zeros(off + rows * (n + pad) + 16, dtype=dtype, device=DEV)
    v = s[off:off + rows * (n + pad)].view(rows, n + pad)[:, :n]
    v.copy_(torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype) if dtype != torch.uint8
            else torch.from_numpy(np.ascontiguousarray(a)).to(DEV))
    return v


INT_CODES = np.array([0x00, 0x38, 0x40, 0x44, 0x48, 0xB8, 0xC0, 0xC4, 0xC8], np.uint8)   # 0, +-1, 2, 3, 4


def integer_case(seed, m, n, k):
    rng = np.random.default_rng(seed)
    dy = rng.integers(-4, 5, size=(k, m)).astype(np.float32)
    q = rng.choice(INT_CODES, size=(k, n))
    sf = rng.integers(126, 129, size=(k, n // 32)).astype(np.uint8)      # 1/2, 1, 2
    return dy, q, sf


CASES = [(1, 32, 1), (8, 32, 7), (16, 64, 64), (127, 96, 33), (128, 128, 128), (130, 160, 65), (256, 256, 192),
         (264, 288, 1), (300, 512, 100), (512, 224, 1000), (1000, 992, 257), (33, 32, 4100), (256, 256, 4096),
         (1024, 2048, 520)]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("layout", [(0, 0, 0, 0), (8, 0, 16, 0), (3, 1, 5, 3)], ids=["packed", "padded", "odd"])
def test_integers(case, layout):
    m, n, k = case
    dy, q, sf = integer_case(1, m, n, k)
    a = strided(dy, torch.bfloat16, layout[0], layout[1])
    b = strided(q, torch.uint8, layout[2], layout[3])
    s = strided(sf, torch.uint8, layout[3], layout[1])
    want = dy.astype(np.float64).T @ ref.dequant(q, sf)
    c = np.random.default_rng(2).integers(-9, 10, size=(m, n)).astype(np.float32)
    D = tg.gemm_wgrad_mxfp8(a, b, s)
    assert np.array_equal(f64(D), want)
    D2 = strided(c, torch.float32, layout[0], layout[1])
    tg.gemm_wgrad_mxfp8(a, b, s, C=D2, D=D2, out_dtype=torch.float32)    # in place
    assert np.array_equal(f64(D2), want + c)
    # bf16 result: the rounding of the exact sum
    Db = tg.gemm_wgrad_mxfp8(a, b, s, C=torch.from_numpy(c).to(DEV).bfloat16(), out_dtype=torch.bfloat16)
    assert np.array_equal(f64(Db), ref.round_to(want + c, "bf16"))


# Grids of 256 x 256 tiles: whole, over one round with the rest cut along K, a
# small grid cut along a long K; the last two rows odd in every size the kernel
# takes (M in its padded rows, N past a tile, K past a K tile).
LARGE = [(3208, 3232, 1), (3208, 3232, 64), (3208, 3232, 65), (3200, 3328, 128), (3201, 3232, 200), (4304, 4096, 2080),
         (1097, 1120, 15500)]


@pytest.mark.parametrize("case", LARGE, ids=str)
@pytest.mark.parametrize("out", OUT)
def test_integers_large_grids(case, out):
    m, n, k = case
    dy, q, sf = integer_case(3, m, n, k)
    a = strided(dy, torch.bfloat16, -m % 8, 0)          # 16-byte rows
    b, s = (torch.from_numpy(t).to(DEV) for t in (q, sf))
    x = torch.from_numpy(ref.dequant(q, sf)).to(DEV)
    c = torch.randint(-9, 10, (m, n), device=DEV).to(OUT[out])
    want = torch.mm(a.double().t().contiguous(), x) + c.double()
    assert want.abs().max() < 2 ** 23                   # halves below 2^23 are fp32 numbers
    D = tg.gemm_wgrad_mxfp8(a, b, s, C=c, out_dtype=OUT[out])
    assert torch.equal(D, want.float().to(OUT[out]))
    assert torch.equal(D, tg.gemm_wgrad_mxfp8(a, b, s, C=c, out_dtype=OUT[out]))
    uncut = tg.gemm_wgrad_mxfp8(a, b, s, C=c, out_dtype=OUT[out], workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    assert torch.equal(D, uncut)


def test_large_grid_leaves_its_surroundings():
    m, n, k = 3208, 3232, 70
    dy, q, sf = integer_case(4, m, n, k)
    A = torch.full((k + 64, m + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    B = torch.full((k + 64, n + 32), 0x7F, dtype=torch.uint8, device=DEV)
    S = torch.full((k + 64, n // 32 + 1), 0xFF, dtype=torch.uint8, device=DEV)
    A[:k, :m], B[:k, :n], S[:k, :n // 32] = (torch.from_numpy(t).to(DEV) for t in (dy, q, sf))
    D = torch.full((m + 3, n + 12), 5.0, device=DEV)
    tg.gemm_wgrad_mxfp8(A[:k, :m], B[:k, :n], S[:k, :n // 32], D=D[:m, :n])
    want = torch.mm(A[:k, :m].double().t().contiguous(), torch.from_numpy(ref.dequant(q, sf)).to(DEV))
    assert torch.equal(D[:m, :n].double(), want)
    D[:m, :n] = 5
    assert (D == 5).all()


@pytest.mark.parametrize("case", [(96, 64, 3000), (520, 480, 1111), (256, 256, 8192), (2048, 1024, 600)], ids=str)
@pytest.mark.parametrize("out", OUT)
def test_random(case, out):
    m, n, k = case
    rng = np.random.default_rng(5)
    dy = torch.from_numpy(rng.standard_normal((k, m)).astype(np.float32)).to(DEV).bfloat16()
    x = torch.from_numpy(rng.standard_normal((k, n)).astype(np.float32)).to(DEV)
    x[:, ::50] *= 100
    q, sf = tg.mxfp8_quantize(x.bfloat16())
    c = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).to(DEV).to(OUT[out])
    D = tg.gemm_wgrad_mxfp8(dy, q, sf, C=c, out_dtype=OUT[out])
    b = ref.dequant(u8(q), u8(sf))
    want, S = f64(dy).T @ b + f64(c), np.abs(f64(dy)).T @ np.abs(b) + np.abs(f64(c))
    bound = (k + 1) * ref.U * S
    if out == "bf16":
        bound = bound + ref.HALF["bf16"] * (np.abs(want) + bound)
    assert (np.abs(f64(D) - want) <= bound).all()


def test_workspace_given_short_or_none():
    """With and without room for cutting K: the same exact sums."""
    m, n, k = 96, 64, 16384
    dy, q, sf = integer_case(7, m, n, k)
    want = dy.astype(np.float64).T @ ref.dequant(q, sf)
    a, b, s = (torch.from_numpy(t).to(DEV) for t in (dy, q, sf))
    a = a.bfloat16()
    need = tg.gemm_wgrad_mxfp8_workspace_bytes(m, n, k)
    assert need > 0
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    for w in (ws[:need], ws[:256], None):
        assert np.array_equal(f64(tg.gemm_wgrad_mxfp8(a, b, s, workspace=w)), want)
    assert (ws[need:] == 0x5A).all()
    D = torch.empty(m, n, device=DEV)
    st = tg.raw.gemm_wgrad_mxfp8(m, n, k, a.data_ptr(), m, b.data_ptr(), n, s.data_ptr(), n // 32, None, 0,
                                 D.data_ptr(), n, 0, None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and np.array_equal(f64(D), want)


def test_no_tokens_and_no_outputs():
    z8 = torch.zeros(0, 64, dtype=torch.uint8, device=DEV)
    zs = torch.zeros(0, 2, dtype=torch.uint8, device=DEV)
    c = torch.randn(40, 64, device=DEV)
    D = tg.gemm_wgrad_mxfp8(torch.zeros(0, 40, dtype=torch.bfloat16, device=DEV), z8, zs, C=c)
    assert torch.equal(D, c)
    D = tg.gemm_wgrad_mxfp8(torch.zeros(0, 40, dtype=torch.bfloat16, device=DEV), z8, zs, D=torch.ones(40, 64, device=DEV))
    assert (D == 0).all()
    D = tg.gemm_wgrad_mxfp8(torch.zeros(5, 0, dtype=torch.bfloat16, device=DEV),
                            torch.zeros(5, 64, dtype=torch.uint8, device=DEV),
                            torch.zeros(5, 2, dtype=torch.uint8, device=DEV))
    assert D.shape == (0, 64)


def test_nan_stays_in_its_columns():
    m, n, k = 200, 320, 100
    dy, q, sf = integer_case(8, m, n, k)
    want = dy.astype(np.float64).T @ ref.dequant(q, sf)
    q[50, 7] = 0x7F                                    # a NaN element: column 7
    sf[3, 5] = 0xFF                                    # a NaN scale: columns 160 .. 191
    D = f64(
        tg.gemm_wgrad_mxfp8(torch.from_numpy(dy).to(DEV).bfloat16(), torch.from_numpy(q).to(DEV),
                            torch.from_numpy(sf).to(DEV)))
    bad = np.zeros(n, bool)
    bad[7] = bad[160:192] = True
    assert np.isnan(D[:, bad]).all() and np.array_equal(D[:, ~bad], want[:, ~bad])


def test_rows_past_the_last_are_not_read():
    """Tokens behind the last (NaN here) and outputs beside the matrix stay out of it."""
    m, n, k = 136, 96, 70
    dy, q, sf = integer_case(9, m, n, k)
    want = dy.astype(np.float64).T @ ref.dequant(q, sf)
    A = torch.full((k + 64, m + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    B = torch.full((k + 64, n + 32), 0x7F, dtype=torch.uint8, device=DEV)
    S = torch.full((k + 64, n // 32 + 1), 0xFF, dtype=torch.uint8, device=DEV)
    A[:k, :m], B[:k, :n], S[:k, :n // 32] = (torch.from_numpy(t).to(DEV) for t in (dy, q, sf))
    D = torch.full((m + 3, n + 16), 5.0, device=DEV)
    tg.gemm_wgrad_mxfp8(A[:k, :m], B[:k, :n], S[:k, :n // 32], D=D[:m, :n])
    assert np.array_equal(f64(D[:m, :n]), want)
    D[:m, :n] = 5
    assert (D == 5).all()


def test_extreme_scales():
    """Scales across bf16's normal range: one token each, so sums are single products."""
    codes = np.arange(12, 246, dtype=np.uint8)         # 2^-115 .. 2^118
    k = codes.size
    for lo in range(0, k, 78):
        sf = codes[lo:lo + 78][:, None]
        q = np.full((sf.shape[0], 32), 0x3C, np.uint8)  # 1.5
        for t in range(0, sf.shape[0], 26):
            D = tg.gemm_wgrad_mxfp8(torch.ones(1, 8, dtype=torch.bfloat16, device=DEV),
                                    torch.from_numpy(q[t:t + 1]).to(DEV), torch.from_numpy(sf[t:t + 1]).to(DEV))
            assert (f64(D) == 1.5 * np.ldexp(1.0, int(sf[t, 0]) - 127)).all()


@pytest.mark.parametrize("shape", [(1, 32), (64, 32), (1, 128), (64, 256)], ids=str)
@pytest.mark.parametrize("lda", [8, 9])
def test_all_scale_codes(shape, lda):
    """Single products at the ends of the scales, over both kernels: exact where bf16 holds the value."""
    k, n = shape
    q = np.zeros((k, n), np.uint8)
    q[0, 0::4], q[0, 1::4] = 0x3C, 0x08                # 1.5, 2^-6
    A = torch.zeros(k, lda, dtype=torch.bfloat16, device=DEV)[:, :8]
    A[0] = 1.0
    for code in (0, 1, 6, 10, 245, 246, 254):
        D = f64(tg.gemm_wgrad_mxfp8(A, torch.from_numpy(q).to(DEV),
                                    torch.full((k, n // 32), code, dtype=torch.uint8, device=DEV)))
        s = np.ldexp(1.0, code - 127)
        assert (D[:, 0::4] == 1.5 * s).all() and (D[:, 1::4] == s / 64).all() and (D[:, 2::4] == 0).all(), code


@pytest.mark.parametrize("case", [(1000, 32, 3001), (4096, 64, 700), (264, 96, 5000), (8, 32, 20000)], ids=str)
@pytest.mark.parametrize("out", OUT)
def test_few_columns(case, out):
    """N below a tile, its scales' rows of one to three bytes and the last one at the end of its storage."""
    m, n, k = case
    dy, q, sf = integer_case(61, m, n, k)
    A, Q = torch.from_numpy(dy.astype(np.float32)).to(DEV).bfloat16(), torch.from_numpy(q).to(DEV)
    S = torch.from_numpy(sf).to(DEV)
    want = dy.astype(np.float64).T @ ref.dequant(q, sf)
    assert np.abs(want).max() < 2 ** 23                 # halves below 2^23 are fp32 numbers
    D = tg.gemm_wgrad_mxfp8(A, Q, S, out_dtype=OUT[out])
    assert np.array_equal(f64(D), want if out == "f32" else ref.round_to(want, "bf16"))


@pytest.mark.parametrize("case", [(1097, 1120, 1700), (4091, 512, 1001), (257, 4096, 2049)], ids=str)
def test_rows_moved_to_16_bytes(case):
    """M that packed rows do not keep on 16 bytes, sizes that copy A into the workspace; and without room for it."""
    m, n, k = case
    dy, q, sf = integer_case(62, m, n, k)
    store = torch.full((k * m + 9,), float("nan"), dtype=torch.bfloat16, device=DEV)
    a = store[1:1 + k * m].view(k, m)                   # NaN on both sides
    a.copy_(torch.from_numpy(dy).to(DEV))
    Q, S = torch.from_numpy(q).to(DEV), torch.from_numpy(sf).to(DEV)
    c = torch.randint(-9, 10, (m, n), device=DEV).float()
    want = torch.mm(a.double().t().contiguous(), torch.from_numpy(ref.dequant(q, sf)).to(DEV)) + c.double()
    assert want.abs().max() < 2 ** 23
    need = tg.gemm_wgrad_mxfp8_workspace_bytes(m, n, k)
    assert need >= k * m * 2
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    D = torch.full((m + 1, n + 3), 5.0, device=DEV)
    tg.gemm_wgrad_mxfp8(a, Q, S, C=c, D=D[:m, :n], workspace=ws[:need])
    assert torch.equal(D[:m, :n].double(), want) and (ws[need:] == 0x5A).all()
    D[:m, :n] = 5
    assert (D == 5).all()
    for short in (need - 1, 0):
        assert torch.equal(tg.gemm_wgrad_mxfp8(a, Q, S, C=c, workspace=ws[:short]).double(), want)


@pytest.mark.parametrize("tiles", range(1, 15))
@pytest.mark.parametrize("shape", [(128, 128), (3328, 3328)], ids=["128x128 tiles", "256x256 tiles"])
def test_every_count_of_k_tiles(shape, tiles):
    """One K range of 1 to 14 K tiles: each way through the unrolled loop and its rest."""
    (m, n), k = shape, 64 * tiles
    g = torch.Generator(DEV).manual_seed(tiles)
    dy = torch.randint(-4, 5, (k, m), device=DEV, generator=g).bfloat16()
    q = torch.from_numpy(INT_CODES).to(DEV)[torch.randint(0, 9, (k, n), device=DEV, generator=g)]
    sf = torch.randint(126, 129, (k, n // 32), device=DEV, generator=g).to(torch.uint8)
    x = q.view(torch.float8_e4m3fn).double() * torch.exp2(sf.double() - 127).repeat_interleave(32, 1)
    want = dy.double().t().contiguous() @ x             # multiples of 1/2 below 2^15
    assert torch.equal(tg.gemm_wgrad_mxfp8(dy, q, sf, workspace=torch.empty(0, dtype=torch.uint8, device=DEV)).double(),
                       want)


@pytest.mark.parametrize("k", [1, 2, 3, 4, 7, 64, 70])
@pytest.mark.parametrize("n", [32, 64, 96, 128, 160, 224, 288])
@pytest.mark.parametrize("pad", [0, 1, 3])
def test_scales_amid_nan_codes(n, k, pad):
    """Scales whose neighbours in memory are NaN codes, before, between and behind their rows."""
    m = 48
    dy, q, sf = integer_case(3, m, n, k)
    s = torch.full((7 + k * (n // 32 + pad) + 9,), 0xFF, dtype=torch.uint8, device=DEV)
    v = s[7:7 + k * (n // 32 + pad)].view(k, n // 32 + pad)[:, :n // 32]
    v.copy_(torch.from_numpy(sf).to(DEV))
    d = tg.gemm_wgrad_mxfp8(torch.from_numpy(dy).to(DEV).bfloat16(), torch.from_numpy(q).to(DEV), v)
    assert np.array_equal(f64(d), dy.astype(np.float64).T @ ref.dequant(q, sf))
