"""gemv_mxfp4 on the GPU: exact on integer values, within |D - D_ref| <= K
2^-24 sum|x w| on random ones, over one to many rows, ragged sizes, rows that
start at any byte, every group width, C and in-place accumulation, scales out
of fp16's range, and NaN scales."""
import numpy as np
import pytest
import torch

import opsref as ref
import tiled_dense_gemm_tile_amd as tg

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
XT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def f64(t):
    return t.detach().double().cpu().numpy()


def strided(a, pad, off):
    rows, n = a.shape
    s = torch.zeros(off + rows * (n + pad) + 16, dtype=a.dtype, device=DEV)
    v = s[off:off + rows * (n + pad)].view(rows, n + pad)[:, :n]
    v.copy_(a)
    return v


def case_of(seed, m, n, k, kb, kind, lo=127, hi=130):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.integers(-4, 5, size=(m, k)).astype(np.float32)).to(DEV).to(XT[kind])
    w = rng.integers(0, 256, size=(n, k // 2), dtype=np.uint8)
    sf = rng.integers(lo, hi, size=(n, -(-k // kb))).astype(np.uint8)
    return x, w, sf


CASES = [(1, 1, 32, 32), (1, 16, 64, 32), (3, 17, 96, 32), (2, 40, 512, 64), (1, 33, 544, 128), (16, 100, 4096, 32),
         (17, 50, 1056, 32), (5, 64, 4128, 4128), (9, 200, 160, 192), (40, 31, 640, 256), (33, 16, 8192, 32),
         (7, 1000, 8224, 32), (64, 48, 4096, 512), (1, 4096, 2048, 32)]


@pytest.mark.parametrize("kind", XT)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_integers(case, kind):
    m, n, k, kb = case
    x, w, sf = case_of(1, m, n, k, kb, kind)
    want = f64(x) @ ref.fp4_weights(w, sf, kb).T        # multiples of 1/2 below 2^23
    assert np.abs(want).max() < 2 ** 22
    W, S = torch.from_numpy(w).to(DEV), torch.from_numpy(sf).to(DEV)
    assert np.array_equal(f64(tg.gemv_mxfp4(x, W, S, kblock=kb)), want)
    c = torch.from_numpy(np.random.default_rng(2).integers(-9, 10, size=(m, n)).astype(np.float32)).to(DEV)
    # rows that start at any element and byte, in-place accumulation
    D = strided(c, 3, 1)
    tg.gemv_mxfp4(strided(x, 5, 1), strided(W, 3, 1), strided(S, 2, 3), kblock=kb, C=D, D=D)
    assert np.array_equal(f64(D), want + f64(c))
    Db = tg.gemv_mxfp4(x, W, S, kblock=kb, C=c.bfloat16(), out_dtype=torch.bfloat16)
    assert np.array_equal(f64(Db), ref.round_to(want + f64(c), "bf16"))


@pytest.mark.parametrize("kind", XT)
@pytest.mark.parametrize("scales", [(116, 122), (100, 145), (60, 190)])
@pytest.mark.parametrize("m", [1, 6, 20])
def test_random(kind, scales, m):
    n, k = 70, 4096
    x, w, sf = case_of(3, m, n, k, 32, kind, *scales)
    x = (torch.randn(m, k, device=DEV, generator=torch.Generator(DEV).manual_seed(4)) * 3).to(XT[kind])
    x[0, ::64] = 6e-8 if kind == "fp16" else 1e-30     # fp16's smallest subnormal
    D = tg.gemv_mxfp4(x, torch.from_numpy(w).to(DEV), torch.from_numpy(sf).to(DEV))
    wv = ref.fp4_weights(w, sf, 32)
    want, S = f64(x) @ wv.T, np.abs(f64(x)) @ np.abs(wv).T
    assert (np.abs(f64(D) - want) <= 2 * k * ref.U * S).all()   # (x in two parts: twice the terms)


# Every path: K ranges (16 rows, 17 rows, few weight rows), blocks per wave and
# waves per block, more blocks than workgroups, every scale width, K off a step.
WIDE = [(16, 4100, 6144, 32), (16, 300, 14336, 128), (20, 1000, 4096, 64), (32, 48, 8192, 32), (1, 512, 16384, 32),
        (3, 9000, 2560, 32), (4, 20000, 1024, 32), (2, 70000, 256, 32), (7, 1111, 4128, 32), (5, 600, 2336, 64),
        (9, 4096, 3360, 128), (1, 2000, 4000, 256), (6, 333, 20000, 4096), (33, 500, 992, 32)]


@pytest.mark.parametrize("kind", XT)
@pytest.mark.parametrize("case", WIDE, ids=str)
def test_integers_wide(case, kind):
    m, n, k, kb = case
    x, w, sf = case_of(11, m, n, k, kb, kind, 127, 129)
    W, S = torch.from_numpy(w).to(DEV), torch.from_numpy(sf).to(DEV)
    want = torch.mm(x.double(), torch.from_numpy(ref.fp4_weights(w, sf, kb)).to(DEV).t().contiguous())
    assert want.abs().max() < 2 ** 22
    c = torch.randint(-9, 10, (m, n), device=DEV).float()
    assert torch.equal(tg.gemv_mxfp4(x, W, S, kblock=kb, C=c).double(), want + c.double())
    b = tg.gemv_mxfp4(x, W, S, kblock=kb, C=c.bfloat16(), out_dtype=torch.bfloat16)
    assert torch.equal(b, (want + c.double()).float().bfloat16())
    # without room for partial sums, and with a workspace whose end is not touched
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    assert torch.equal(tg.gemv_mxfp4(x, W, S, kblock=kb, C=c, workspace=none).double(), want + c.double())
    need = tg.gemv_mxfp4_workspace_bytes(m, n, k)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    D = torch.full((m + 1, n + 7), 5.0, device=DEV)
    tg.gemv_mxfp4(x, W, S, kblock=kb, C=c, D=D[:m, :n], workspace=ws[:need])
    assert torch.equal(D[:m, :n].double(), want + c.double()) and (ws[need:] == 0x5A).all()
    D[:m, :n] = 5
    assert (D == 5).all()


def test_x_in_two_parts_over_the_staged_path():
    """fp16 X against scales out of fp16's range, K past a step and wide enough for every wave."""
    for k in (4096, 4128):
        x, w, sf = case_of(12, 5, 100, k, 32, "fp16", 127, 129)
        sf[:, 3::7] = 150                              # 2^23
        wv = ref.fp4_weights(w, sf, 32)
        want, S = f64(x) @ wv.T, np.abs(f64(x)) @ np.abs(wv).T
        D = f64(tg.gemv_mxfp4(x, torch.from_numpy(w).to(DEV), torch.from_numpy(sf).to(DEV)))
        assert (np.abs(D - want) <= 2 * k * ref.U * S).all()


def test_fp16_weights_stay_exact_at_the_range_border():
    """Single products at scales around fp16's: subnormal and large weights."""
    for code in (100, 103, 104, 105, 112, 113, 114, 139, 140, 141, 150):
        w = np.arange(256, dtype=np.uint8).reshape(16, 16)
        sf = np.full((16, 1), code, np.uint8)
        for j in range(0, 32, 5):
            x = torch.zeros(1, 32, dtype=torch.float16, device=DEV)
            x[0, j] = 1.0
            D = f64(tg.gemv_mxfp4(x, torch.from_numpy(w).to(DEV), torch.from_numpy(sf).to(DEV)))
            assert np.array_equal(D[0], ref.fp4_weights(w, sf, 32)[:, j]), code


def test_fp16_extremes():
    """The largest and smallest fp16 numbers, and infinities that stay in their row."""
    k, n = 64, 16
    w = np.full((n, k // 2), 0x22, np.uint8)           # ones
    for code in (127, 160):
        sf = np.full((n, 2), code, np.uint8)
        x = torch.zeros(3, k, dtype=torch.float16, device=DEV)
        x[0, 5], x[1, 40], x[2, 3] = 65504.0, float("inf"), 2.0 ** -24
        D = f64(tg.gemv_mxfp4(x, torch.from_numpy(w).to(DEV), torch.from_numpy(sf).to(DEV)))
        s = 2.0 ** (code - 127)
        assert (D[0] == 65504.0 * s).all() and (D[1] == np.inf).all() and (D[2] == 2.0 ** -24 * s).all()


def test_nan_scale_stays_in_its_column():
    x, w, sf = case_of(6, 4, 50, 256, 32, "bf16")
    want = f64(x) @ ref.fp4_weights(w, sf, 32).T
    sf[21, 3] = 0xFF
    D = f64(tg.gemv_mxfp4(x, torch.from_numpy(w).to(DEV), torch.from_numpy(sf).to(DEV)))
    keep = np.arange(50) != 21
    assert np.isnan(D[:, 21]).all() and np.array_equal(D[:, keep], want[:, keep])


def test_nothing_past_the_matrices():
    """NaN scales, codes and X behind the last row and column stay out; D's surroundings stay as they are."""
    m, n, k = 3, 37, 96
    x, w, sf = case_of(7, m, n, k, 32, "bf16")
    want = f64(x) @ ref.fp4_weights(w, sf, 32).T
    X = torch.full((m + 20, k + 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    W = torch.full((n + 20, k // 2 + 64), 0x77, dtype=torch.uint8, device=DEV)
    S = torch.full((n + 20, k // 32 + 16), 0xFF, dtype=torch.uint8, device=DEV)
    X[:m, :k], W[:n, :k // 2], S[:n, :3] = x, torch.from_numpy(w).to(DEV), torch.from_numpy(sf).to(DEV)
    D = torch.full((m + 2, n + 9), 5.0, device=DEV)
    tg.gemv_mxfp4(X[:m, :k], W[:n, :k // 2], S[:n, :3], D=D[:m, :n])
    assert np.array_equal(f64(D[:m, :n]), want)
    D[:m, :n] = 5
    assert (D == 5).all()


def test_no_k_and_no_rows():
    c = torch.randn(3, 20, device=DEV)
    z = torch.zeros(20, 0, dtype=torch.uint8, device=DEV)
    x = torch.zeros(3, 0, dtype=torch.bfloat16, device=DEV)
    assert torch.equal(tg.gemv_mxfp4(x, z, z, C=c), c)
    assert (tg.gemv_mxfp4(x, z, z, D=torch.ones(3, 20, device=DEV)) == 0).all()
    w = torch.zeros(20, 16, dtype=torch.uint8, device=DEV)
    s = torch.zeros(20, 1, dtype=torch.uint8, device=DEV)
    assert tg.gemv_mxfp4(torch.zeros(0, 32, dtype=torch.bfloat16, device=DEV), w, s).shape == (0, 20)


def test_agrees_with_the_block_scaled_product():
    """The same weights through gemm_mxfp4, with X that e2m1 holds exactly."""
    n, k = 96, 512
    _, w, sf = case_of(9, 16, n, k, 32, "bf16")
    xc = np.random.default_rng(10).integers(0, 256, size=(16, k // 2), dtype=np.uint8)
    one = np.full((16, k // 32), 127, np.uint8)
    X = torch.from_numpy(ref.fp4_weights(xc, one, 32).astype(np.float32)).to(DEV).bfloat16()
    W, S = torch.from_numpy(w).to(DEV), torch.from_numpy(sf).to(DEV)
    A = tg.gemm_mxfp4(torch.from_numpy(xc).to(DEV), torch.from_numpy(one).to(DEV), W, S)
    assert torch.equal(tg.gemv_mxfp4(X, W, S), A)


@pytest.mark.parametrize("kind", XT)
@pytest.mark.parametrize("case", [(500, 16400, 1056, 32), (2400, 500, 14336, 128)], ids=str)
def test_rows_in_several_passes(case, kind):
    """More rows than the partial sums of one pass hold: whole passes and a shorter last one."""
    m, n, k, kb = case
    x, w, sf = case_of(13, m, n, k, kb, kind, 127, 129)
    W, S = torch.from_numpy(w).to(DEV), torch.from_numpy(sf).to(DEV)
    need = tg.gemv_mxfp4_workspace_bytes(m, n, k)
    splits = -(-k // 1024)
    assert 0 < need < splits * m * n * 4 and need <= 64 << 20
    want = torch.mm(x.double(), torch.from_numpy(ref.fp4_weights(w, sf, kb)).to(DEV).t().contiguous())
    assert want.abs().max() < 2 ** 22
    c = torch.randint(-9, 10, (m, n), device=DEV).float()
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    D = torch.full((m + 1, n + 3), 5.0, device=DEV)
    D[:m, :n] = c
    tg.gemv_mxfp4(x, W, S, kblock=kb, C=D[:m, :n], D=D[:m, :n], workspace=ws[:need])
    assert torch.equal(D[:m, :n].double(), want + c.double()) and (ws[need:] == 0x5A).all()
    D[:m, :n] = 5
    assert (D == 5).all()
    b = tg.gemv_mxfp4(x, W, S, kblock=kb, C=c.bfloat16(), out_dtype=torch.bfloat16)
    assert torch.equal(b, (want + c.double()).float().bfloat16())


@pytest.mark.parametrize("kind", XT)
@pytest.mark.parametrize("k", [32, 256])
def test_all_scale_codes(kind, k):
    """One weight of each row against 1.0: exact from 2^-127 up; infinite past bf16's range."""
    w = np.full((3, k // 2), 0x21, np.uint8)           # 0.5, 1
    w[1], w[2] = 0x75, 0                               # 3, 6; zeros
    x = torch.zeros(2, k, dtype=XT[kind], device=DEV)
    x[0, 0], x[1, 1] = 1.0, 1.0
    for code in (0, 1, 2, 9, 103, 104, 135, 136, 245, 252, 253, 254):
        D = f64(tg.gemv_mxfp4(x, torch.from_numpy(w).to(DEV),
                              torch.full((3, k // 32), code, dtype=torch.uint8, device=DEV)))
        s = np.ldexp(1.0, code - 127)
        assert np.array_equal(D[0, [0, 2]], [0.5 * s, 0]) and np.array_equal(D[1, [0, 2]], [s, 0]), code
        if code <= 252:
            assert np.array_equal(D[:, 1], [3 * s, 6 * s]), code
        else:
            assert not np.isfinite(D[:, 1]).any(), code


@pytest.mark.parametrize("kind", XT)
@pytest.mark.parametrize("k", [32, 256])
@pytest.mark.parametrize("m", [1, 20])
def test_weights_past_bf16_are_infinite(kind, k, m):
    """Non-zero x against one weight at or past 2^128 and zeros: an infinity of the product's sign, with x that bf16
    holds and x that it does not; the largest finite weights of the same scales stay exact."""
    x = torch.tensor([1.0, 0.1, -3.1416, 2.0 ** -10] * (k // 4), device=DEV).to(XT[kind]).repeat(m, 1)
    for code, over, finite in ((253, (4, 6), 3), (254, (2, 3, 4, 6), 1.5)):
        codes = [list(ref.E2M1).index(v) for v in over]
        rows = [(c ^ s, at) for c in codes for s in (0, 8) for at in range(4)]
        w = np.zeros((len(rows) + 4, k // 2), np.uint8)
        for i, (c, at) in enumerate(rows):
            w[i, at // 2] = c << (4 * (at % 2))
        for at in range(4):
            w[len(rows) + at, at // 2] = list(ref.E2M1).index(finite) << (4 * (at % 2))
        S = torch.full((len(w), k // 32), code, dtype=torch.uint8, device=DEV)
        D = f64(tg.gemv_mxfp4(x, torch.from_numpy(w).to(DEV), S))
        xv = f64(x)
        for i, (c, at) in enumerate(rows):
            assert (D[:, i] == np.sign(xv[:, at]) * (np.inf if c < 8 else -np.inf)).all(), (code, c, at)
        # (in fp32: 3.1416 * 1.5 * 2^127 is past its range)
        with np.errstate(over="ignore"):
            want = (xv[:, :4] * finite * np.ldexp(1.0, code - 127)).astype(np.float32).astype(np.float64)
        assert np.array_equal(D[:, len(rows):], want), code
