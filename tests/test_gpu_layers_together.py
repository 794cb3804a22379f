"""The feed-forward layer's operators as they are used together: a training
step with clipped gradients, a serving step in 8-bit integers and one of a
single token, as captured graphs replayed with new inputs and on other
streams; and what the binding refuses on the GPU."""
import math

import pytest
import torch

import layersref as ref
import tiled_dense_gemm_tile_amd as tg
from layersref import DEV, U, act, half, rand, within
from opsref import HALF

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


def training_step(x, w, Wg, Wu, Wd, dy, top=1.0, grads=None):
    """y = (silu(n Wg^T) * (n Wu^T)) Wd^T, n = norm(x); gradients of x and all weights, these clipped in place."""
    n, h, rstd = tg.rmsnorm(x, w, EPS)
    a, g, u = tg.gemm_glu(n, Wg, Wu, keep=True)
    y = tg.gemm_bf16(a, Wd, out_dtype=BF)
    dWd = tg.gemm_bf16(dy.t(), a.t(), out_dtype=F32)
    da = tg.gemm_bf16(dy, Wd.t(), out_dtype=BF)
    dn, dWg, dWu = tg.gemm_glu_backward(da, g, u, n, Wg, Wu, grad_dtype=F32)
    dx, dw = tg.rmsnorm_backward(dn, h, w, rstd)
    grads = [dWd, dWg, dWu, dw]
    norm = tg.clip_grads(grads, top)
    return y, dx, norm, *grads


def layer(T, d, f, seed=0):
    x, w = rand(seed + 1, T, d), rand(seed + 2, d, scale=0.1) + 1
    return (x, w, rand(seed + 3, f, d, scale=d ** -0.5), rand(seed + 4, f, d, scale=d ** -0.5),
            rand(seed + 5, d, f, scale=f ** -0.5), rand(seed + 6, T, d, scale=0.1))


def test_training_step():
    """Gradients against autograd's in 64 bits on the same inputs: every intermediate is rounded to bf16 (2^-8 of a
    value at most), nine times on the longest way (n, g, u, a, da, dg or du, dn, dx, its input), and errors of many
    terms add like their norms."""
    T, d, f = 200, 256, 384
    x, w, Wg, Wu, Wd, dy = layer(T, d, f)
    y, dx, norm, *grads = training_step(x, w, Wg, Wu, Wd, dy, top=1e9)
    leaves = [t.double().requires_grad_() for t in (x, w, Wg, Wu, Wd)]
    lx, lw, lg, lu, ld = leaves
    n = lx * torch.rsqrt((lx * lx).mean(1, keepdim=True) + EPS) * lw
    g = n @ lg.t()
    out = (g * torch.sigmoid(g) * (n @ lu.t())) @ ld.t()
    out.backward(dy.double())
    for got, want in ((y, out.detach()), (dx, lx.grad), (grads[0], ld.grad), (grads[1], lg.grad), (grads[2], lu.grad), (grads[3], lw.grad)):
        assert float((got.double() - want).norm()) <= 9 * HALF["bf16"] * float(want.norm())
    want = math.sqrt(sum(float((t.double() ** 2).sum()) for t in grads))
    assert abs(float(norm) - want) <= 2 * U * want
    # clipped: the norm is the bound, to the factor's roundings
    clipped = training_step(x, w, Wg, Wu, Wd, dy, top=0.25 * want)
    assert abs(float(tg.grad_norm(clipped[3:])) - 0.25 * want) <= 8 * U * want


def serving_step(x, w, Wq, Ws, Dq, Ds):
    """Two projections in 8-bit integers behind a norm, the second onto the residual stream."""
    n, h, _ = tg.rmsnorm(x, w, EPS)
    q, s = tg.int8_quantize(n)
    a = tg.gemm_int8(q, s, Wq, Ws, out_dtype=BF)
    q2, s2 = tg.int8_quantize(a)
    return tg.gemm_int8(q2, s2, Dq, Ds, C=h, out_dtype=BF), q, s, a, q2, s2, h


@pytest.mark.parametrize("T", [1, 16, 100])
def test_serving_step(T):
    d, f = 512, 704
    x, w = rand(1, T, d), rand(2, d, scale=0.1) + 1
    Wq, Ws = tg.int8_quantize(rand(3, f, d, scale=d ** -0.5))
    Dq, Ds = tg.int8_quantize(rand(4, d, f, scale=f ** -0.5))
    y, q, s, a, q2, s2, h = serving_step(x, w, Wq, Ws, Dq, Ds)
    for got, A, SA, B, SB, C in ((a, q, s, Wq, Ws, None), (y, q2, s2, Dq, Ds, h)):
        want = (A.double() @ B.double().t()) * SA.double()[:, None] * SB.double()
        bound = 3 * U * want.abs()
        if C is not None:
            want = want + C.double()
            bound = bound + U * (want.abs() + bound)
        within(got, want, half(want, bound, BF))


def replayed(step, inputs, fresh, rounds=4):
    """The step as a graph, replayed with new inputs and eager work between, against the eager step each time."""
    static = [t.clone() for t in inputs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*static)
    for i in range(rounds):
        new = fresh(i)
        for s, n in zip(static, new):
            s.copy_(n)
        graph.replay()
        want = step(*new)
        torch.cuda.synchronize()
        for o, v in zip(outs, want):
            assert torch.equal(o, v), "replay %d" % i


def test_training_step_captured():
    T, d, f = 304, 320, 504                            # (gemm_bf16 of MN-contiguous operands takes rows of 16 bytes)
    make = lambda i: layer(T, d, f, 100 * (i + 1))
    replayed(training_step, make(9), make)


def test_large_step_captured():
    """The kernels of large grids."""
    m, f, k = 2100, 2100, 520
    make = lambda i: [rand(50 * i + j, m, f) for j in range(3)] + [rand(50 * i + 3, m, k), rand(50 * i + 4, f, k), rand(50 * i + 5, f, k)]

    def step(dh, g, u, x, wg, wu):
        h = tg.gemm_glu(x, wg, wu)
        return (h, *tg.gemm_glu_backward(dh, g, u, x, wg, wu))

    replayed(step, make(9), make)


@pytest.mark.parametrize("T", [1, 40])
def test_serving_step_captured(T):
    d, f = 512, 704
    w = rand(2, d, scale=0.1) + 1
    Wq, Ws = tg.int8_quantize(rand(3, f, d, scale=d ** -0.5))
    Dq, Ds = tg.int8_quantize(rand(4, d, f, scale=f ** -0.5))
    replayed(lambda x: serving_step(x, w, Wq, Ws, Dq, Ds), [rand(1, T, d)], lambda i: [rand(70 + i, T, d)])


def test_other_stream():
    """Work on a stream of its own, whose inputs that stream makes, while another stream is busy."""
    T, d, f = 400, 512, 600
    want = training_step(*layer(T, d, f))
    side = torch.cuda.Stream()
    busy = torch.randn(2048, 2048, device=DEV)
    torch.cuda.synchronize()
    for _ in range(4):
        busy = busy @ busy * 1e-3
    with torch.cuda.stream(side):
        got = training_step(*layer(T, d, f))
    side.synchronize()
    for g, v in zip(got, want):
        assert torch.equal(g, v)


def test_two_calls_at_once():
    """Two streams, each with its own results and workspace."""
    a = [layer(304, 256, 704, s) for s in (0, 50)]
    want = [training_step(*t) for t in a]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for s, t in zip(streams, a):
        with torch.cuda.stream(s):
            got.append(training_step(*t))
    torch.cuda.synchronize()
    for g, v in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(g, v))


def test_same_values_same_bits():
    x, wg, wu = rand(1, 2100, 264), rand(2, 2100, 264), rand(3, 2100, 264)
    first = tg.gemm_glu(x, wg, wu, keep=True)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, tg.gemm_glu(x, wg, wu, keep=True)))


def test_workspace_given():
    m, f, k = 100, 130, 70
    a = [rand(i, m, f) for i in range(3)] + [rand(3, m, k), rand(4, f, k), rand(5, f, k)]
    need = tg.gemm_glu_backward_workspace_bytes(m, f, k)
    guard = torch.full((need + 512,), 171, dtype=torch.uint8, device=DEV)
    want = tg.gemm_glu_backward(*a)
    got = tg.gemm_glu_backward(*a, workspace=guard[:need])
    assert all(torch.equal(p, q) for p, q in zip(got, want)) and bool((guard[need:] == 171).all())
    with pytest.raises(tg.GemmError) as e:
        tg.gemm_glu_backward(*a, workspace=guard[:need - 1])
    assert e.value.status == 7
    grads = [rand(i, 9000 * i + 1) for i in range(1, 150)]
    need = tg.grad_workspace_bytes(len(grads))
    guard = torch.full((need + 512,), 171, dtype=torch.uint8, device=DEV)
    assert torch.equal(tg.grad_norm(grads, workspace=guard[:need]), tg.grad_norm(grads)) and bool((guard[need:] == 171).all())


def test_refusals():
    x, w, h = rand(1, 8, 64), rand(2, 16, 64), rand(3, 8, 16)
    q, s = tg.int8_quantize(x)
    wq, ws = tg.int8_quantize(w)
    value = [lambda: tg.gemm_glu(x, w, w, act="tanh"), lambda: tg.gemm_glu(x, w, w[:, :32]), lambda: tg.gemm_glu(x, w, w[:8]),
             lambda: tg.gemm_glu(x, w.t().contiguous().t(), w), lambda: tg.gemm_glu(x, w, w, H=h[:4]),
             lambda: tg.gemm_glu(x, w, w.cpu()), lambda: tg.gemm_glu_backward(h, h, h, x, w, w, Cg=w),
             lambda: tg.gemm_glu_backward(h, h, h, x, w, w, input_grad=False, dX=x),
             lambda: tg.gemm_glu_backward(h, h, h, x, w, w, weight_grad=False, dWg=w),
             lambda: tg.gemm_int8(q, s[:4], wq, ws), lambda: tg.gemm_int8(q, s, wq[:, :32], ws),
             lambda: tg.gemm_int8(q, s, wq, ws, C=torch.zeros(5, device=DEV)), lambda: tg.int8_quantize(x, S=s[:3]),
             lambda: tg.clip_grads([x, x], 1.0), lambda: tg.clip_grads([x[:, :32]], 1.0), lambda: tg.clip_grads([x], 1.0, out=[]),
             lambda: tg.clip_grads([x], 1.0, out=[h]), lambda: tg.clip_grads([x, w], 1.0, out=[x[:4], w]),
             lambda: tg.clip_grads([x.t()], 1.0, out=[x.t().contiguous()]), lambda: tg.clip_grads([x], 1.0, given=s),
             lambda: tg.clip_grads([x], 1.0, given=s[:1], norm=s[1:2]), lambda: tg.grad_norm([x, w.cpu()]), lambda: tg.grad_norm([])]
    for f in value:
        with pytest.raises(ValueError):
            f()
    kind = [lambda: tg.gemm_glu(x, w.half(), w), lambda: tg.gemm_glu(x, w, w, H=h.float()),
            lambda: tg.gemm_glu_backward(h, h.half(), h, x, w, w), lambda: tg.gemm_glu_backward(h, h, h, x, w, w, grad_dtype=FP),
            lambda: tg.gemm_int8(q, s, wq.float(), ws), lambda: tg.gemm_int8(q, s.half(), wq, ws),
            lambda: tg.gemm_int8(q, s, wq, ws, out_dtype=torch.int32), lambda: tg.gemm_int8(q, s, wq, ws, C=h, out_dtype=F32),
            lambda: tg.grad_norm([q])]
    for f in kind:
        with pytest.raises(TypeError):
            f()
    status = [lambda: tg.gemm_glu(x, w, w, G=h, H=h), lambda: tg.gemm_glu(x[:, :16], w[:, :16], w[:, :16], H=x[:, 16:32]),
              lambda: tg.clip_grads([x], -1.0), lambda: tg.clip_grads([x], float("nan"))]
    for f in status:
        with pytest.raises(tg.GemmError):
            f()
