"""The operators as they are used together: a training step of a block-scaled
linear layer behind a norm, a decode step with 4-bit weights, and both as
captured graphs replayed with new inputs."""
import numpy as np
import pytest
import torch

import opsref as ref
import tiled_dense_gemm_tile_amd as tg

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
EPS = 1e-5


def f64(t):
    return t.detach().double().cpu().numpy()


def u8(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def rand(seed, *shape, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def training_step(x, r, w, Wq, Ws, Wb, dy, dh):
    """y = norm(x + r) W^T in block-scaled fp8; gradients of x, w and W."""
    q, sf, h, rstd = tg.rmsnorm_mxfp8(x, w, EPS, residual=r)
    y = tg.gemm_mxfp8(q, sf, Wq, Ws, out_dtype=torch.bfloat16)
    dW = tg.gemm_wgrad_mxfp8(dy, q, sf)
    dn = tg.gemm_bf16(dy, Wb.t(), out_dtype=torch.bfloat16)
    dx, dw = tg.rmsnorm_backward(dn, h, w, rstd, dH=dh)
    return y, dW, dn, dx, dw, q, sf, h, rstd


def test_training_step():
    T, n, m = 400, 512, 768
    x, r, w = rand(1, T, n), rand(2, T, n), rand(3, n, scale=0.1) + 1
    Wb = rand(4, m, n, scale=0.05)
    Wq, Ws = tg.mxfp8_quantize(Wb)
    dy, dh = rand(5, T, m, scale=0.01), rand(6, T, n, scale=0.01)
    y, dW, dn, dx, dw, q, sf, h, rstd = training_step(x, r, w, Wq, Ws, Wb, dy, dh)
    a, b = ref.dequant(u8(q), u8(sf)), ref.dequant(u8(Wq), u8(Ws))
    want, S = a @ b.T, np.abs(a) @ np.abs(b).T
    bound = n * ref.U * S + 1e-6
    assert (np.abs(f64(y) - want) <= bound + ref.HALF["bf16"] * (np.abs(want) + bound)).all()
    want, S = f64(dy).T @ a, np.abs(f64(dy)).T @ np.abs(a)
    assert (np.abs(f64(dW) - want) <= T * ref.U * S).all()
    # gradients of the layer: the norm's backward on the input gradient that the product handed on
    wdx, wdw, ag, au, adw = ref.norm_backward(f64(dn), f64(h), f64(w), f64(rstd), f64(dh))
    bound = 4 * ref.U * ag + (n / 64 + 41) * ref.U * au + 2 * ref.U * np.abs(wdx)
    assert (np.abs(f64(dx) - wdx) <= bound + ref.HALF["bf16"] * (np.abs(wdx) + bound)).all()
    assert (np.abs(f64(dw) - wdw) <= (T / 64 + 67) * ref.U * adw).all()
    # the 8-bit operand is the norm's result to half a step of e4m3
    yn, _ = ref.norm(f64(h), f64(w), EPS)
    assert np.linalg.norm(a - yn) <= 2.0 ** -4 * np.linalg.norm(yn)


def test_accumulated_weight_gradient():
    """Two micro-batches into one gradient equal the joined batch's, in the sums' bound."""
    dy, x = rand(7, 600, 160), rand(8, 600, 96)
    q, sf = tg.mxfp8_quantize(x)
    D = tg.gemm_wgrad_mxfp8(dy[:250], q[:250], sf[:250])
    tg.gemm_wgrad_mxfp8(dy[250:], q[250:], sf[250:], C=D, D=D)
    a = ref.dequant(u8(q), u8(sf))
    assert (np.abs(f64(D) - f64(dy).T @ a) <= 601 * ref.U * (np.abs(f64(dy)).T @ np.abs(a))).all()


def decode(x, r, w, W1, S1, W2, S2):
    """norm(x + r) through two 4-bit projections, the second onto the residual stream."""
    y, h, _ = tg.rmsnorm(x, w, EPS, residual=r)
    u = tg.gemv_mxfp4(y, W1, S1, out_dtype=torch.bfloat16)
    return tg.gemv_mxfp4(u, W2, S2, kblock=128, C=h, out_dtype=torch.bfloat16), u, y, h


def weights(seed, n, k, kb):
    rng = np.random.default_rng(seed)
    return (torch.from_numpy(rng.integers(0, 256, size=(n, k // 2), dtype=np.uint8)).to(DEV),
            torch.from_numpy(rng.integers(117, 121, size=(n, k // kb)).astype(np.uint8)).to(DEV))


def test_decode_step():
    n, f = 512, 1280
    x, r, w = rand(9, 3, n), rand(10, 3, n), rand(11, n, scale=0.1) + 1
    W1, W2 = weights(12, f, n, 32), weights(13, n, f, 128)
    out, u, y, h = decode(x, r, w, *W1, *W2)
    for got, a, (W, S), kb, c in ((u, y, W1, 32, 0.0), (out, u, W2, 128, f64(h))):
        v = ref.fp4_weights(W.cpu().numpy(), S.cpu().numpy(), kb)
        want, mag = f64(a) @ v.T + c, np.abs(f64(a)) @ np.abs(v).T + np.abs(c)
        bound = (v.shape[1] + 1) * ref.U * mag
        assert (np.abs(f64(got) - want) <= bound + ref.HALF["bf16"] * (np.abs(want) + bound)).all()


def replayed(step, inputs, other):
    """`step` captured on `inputs`, replayed after they are overwritten with
    each of `other` in turn; every replay against the eager result."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(*inputs)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(*inputs)
    for new in other:
        for a, b in zip(inputs, new):
            a.copy_(b)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = step(*[t.clone() for t in new])
        for a, b in zip(out, want):
            assert torch.equal(a.view(torch.uint8) if a.dtype.itemsize == 1 else a,
                               b.view(torch.uint8) if b.dtype.itemsize == 1 else b)


def test_training_step_captured():
    T, n, m = 300, 256, 384

    def inputs(s):
        Wb = rand(s + 3, m, n, scale=0.05)
        return [rand(s, T, n), rand(s + 1, T, n), rand(s + 2, n, scale=0.1) + 1, *tg.mxfp8_quantize(Wb), Wb,
                rand(s + 4, T, m, scale=0.01), rand(s + 5, T, n, scale=0.01)]

    ins = inputs(20)
    replayed(training_step, ins, [inputs(40), inputs(60), inputs(80)])


def test_decode_step_captured():
    n, f = 256, 640

    def inputs(s):
        return [rand(s, 2, n), rand(s + 1, 2, n), rand(s + 2, n, scale=0.1) + 1, *weights(s, f, n, 32),
                *weights(s + 1, n, f, 128)]

    replayed(decode, inputs(20), [inputs(40), inputs(60), inputs(80)])


def test_calls_on_another_stream():
    x, w = rand(90, 700, 1024), rand(91, 1024)
    want = tg.rmsnorm_mxfp8(x, w, EPS)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = tg.rmsnorm_mxfp8(x, w, EPS)
        dW = tg.gemm_wgrad_mxfp8(rand(92, 700, 64), got[0], got[1])
    s.synchronize()
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8))
    assert torch.equal(dW, tg.gemm_wgrad_mxfp8(rand(92, 700, 64), want[0], want[1]))


def test_the_last_token_of_a_long_batch_of_one():
    """x[:, -1] is one row whose stride is the whole batch: as good as a packed row."""
    n, m = 4096, 96
    x = rand(30, 1, 2100, n)
    last, row = x[:, -1], x[0, -1:].clone()
    assert last.stride(0) * 2 >= 8 << 20
    w = rand(31, n, scale=0.1) + 1
    W = torch.randint(0, 256, (m, n // 2), device=DEV, generator=torch.Generator(DEV).manual_seed(32)).to(torch.uint8)
    S = torch.full((m, n // 32), 120, dtype=torch.uint8, device=DEV)
    assert torch.equal(tg.gemv_mxfp4(last, W, S), tg.gemv_mxfp4(row, W, S))
    q, sf = tg.mxfp8_quantize(last)
    for a, b in zip((q, sf), tg.mxfp8_quantize(row)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(tg.gemm_wgrad_mxfp8(last, q, sf), tg.gemm_wgrad_mxfp8(row, q, sf))
    y = tg.rmsnorm(row, w, EPS)[0]
    out = torch.zeros_like(x)
    tg.rmsnorm(last, w, EPS, Y=out[:, -1])              # and so for results
    assert torch.equal(out[:, -1], y) and (out[:, :-1] == 0).all()
    D = torch.zeros(1, 40000, m, device=DEV)
    tg.gemv_mxfp4(row, W, S, D=D[:, -1])
    assert torch.equal(D[:, -1], tg.gemv_mxfp4(row, W, S)) and (D[:, :-1] == 0).all()
