"""Edges of the feed-forward layer's operators that sizes and random inputs do
not reach: scales next to the smallest one, infinite bounds, many tensors."""
import pytest
import torch

import layersref as ref
import tiled_dense_gemm_tile_amd as tg
from layersref import DEV, KIND, rand
from tiled_dense_gemm_tile_amd import layers, ops

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


# ---- codes of rows whose scale is next to 2^-126 ----------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF], ids=KIND.get)
@pytest.mark.parametrize("binade", [-128, -127, -126, -125, -124, -100])
def test_quantize_codes_of_tiny_rows(binade, dtype):
    """Elements at the codes' borders and their neighbours, in rows whose scale lies in [2^binade, 2^(binade + 1)): the
    remainder at a border of a scale just over 2^-126 is below the least subnormal."""
    g = torch.Generator(DEV).manual_seed(11)
    top = ((torch.rand(200, 1, generator=g, device=DEV) + 1) * 127 * 2.0 ** binade).to(dtype).float()
    scale = ref.quantize(top)[1].double()[:, None]
    k = torch.arange(-126, 126, device=DEV, dtype=torch.float64) + 0.5
    near = (k * scale).to(dtype)
    steps = near.view(torch.int32 if dtype == F32 else torch.int16)
    x = torch.cat([top.to(dtype), near, (steps + 1).view(dtype), (steps - 1).view(dtype)], 1)
    # (a neighbour of a border past the row's largest number would change its scale)
    x = torch.where(x.float().abs() <= top, x, torch.zeros_like(x))
    q, s = tg.int8_quantize(x)
    wq, ws = ref.quantize(x)
    assert torch.equal(s, ws)
    assert torch.equal(q, wq), "%d codes off" % int((q != wq).sum())


@pytest.mark.parametrize("dtype", [F32, BF], ids=KIND.get)
def test_quantize_remainder_below_the_least_subnormal(dtype):
    """A quotient of 63.5 - 3.4e-8, whose remainder is -2^-150: no tie."""
    x = torch.tensor([[float.fromhex("0x1.bcp-119"), float.fromhex("0x1.bcp-120")]], device=DEV).to(dtype)
    q, s = tg.int8_quantize(x)
    assert q.tolist() == [[127, 63]] and torch.equal(s, ref.quantize(x)[1])


# ---- memory next to each other -----------------------------------------------------------

def test_norm_next_to_the_gradients():
    """Gradients that are views of each other, the norm between two of them, the workspace behind."""
    room = tg.grad_workspace_bytes(3)
    flat = rand(1, 1 << 18, dtype=F32)
    grads, norm = [flat[:1001], flat[500:1001], flat[1002:30000]], flat[1001:1002]
    want = torch.linalg.vector_norm(torch.cat(grads), dtype=torch.float64)
    ws = flat[30016:].view(torch.uint8)[:room + 64]
    ws = ws[-ws.data_ptr() % 256:][:room]
    got = tg.grad_norm(grads, norm=norm, workspace=ws)
    assert abs(float(got) - float(want)) <= 2.0 ** -23 * float(want)
    for over in (dict(norm=flat[1000:1001]), dict(norm=ws[:4].view(F32), workspace=ws),
                 dict(workspace=flat.view(torch.uint8)[:room])):
        with pytest.raises(tg.GemmError):
            tg.grad_norm(grads, **over)


# ---- an infinite bound ------------------------------------------------------------------

def test_clip_by_an_infinite_bound():
    """The norm alone: gradients stay, whatever the norm is, unless that is a NaN."""
    for bad, want in ((None, None), (float("inf"), "same"), (float("nan"), "nan")):
        g = [rand(1, 9000, dtype=BF), rand(2, 70001, dtype=F32)]
        if bad is not None:
            g[1][69999] = bad
        keep = [t.clone() for t in g]
        out = [torch.full_like(t, 7) for t in g]
        n = tg.clip_grads(g, float("inf"), out=out)
        given = tg.clip_grads([t.clone() for t in g], float("inf"), given=n)
        assert given is n and torch.equal(n, tg.grad_norm(g)) or want == "nan"
        n2 = tg.clip_grads(g, float("inf"))
        assert torch.equal(n, n2) or want == "nan"
        for t, k, o in zip(g, keep, out):
            if want == "nan":
                assert bool(t.isnan().all()) and bool(o.isnan().all())
            else:
                assert torch.equal(t, k) and torch.equal(o, k)


# ---- many tensors -----------------------------------------------------------------------

def milliseconds(f, rounds=5):
    f()
    best = float("inf")
    for _ in range(rounds):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


def test_clip_of_many_tensors_costs_its_parts():
    """Thousands of tensors are scaled over many launches: the norm is computed once for all of them, so that the whole
    call costs about what the norm and a scaling by a given norm do."""
    n, size = 6000, 1 << 17
    flat = rand(1, n * size, dtype=BF)
    grads = [flat[i * size:(i + 1) * size] for i in range(n)]
    out = torch.empty_like(flat)
    outs = [out[i * size:(i + 1) * size] for i in range(n)]
    norm = tg.grad_norm(grads)
    whole = milliseconds(lambda: tg.clip_grads(grads, 1.0, out=outs))
    parts = milliseconds(lambda: tg.grad_norm(grads)) + milliseconds(lambda: tg.clip_grads(grads, 1.0, out=outs, given=norm))
    print("clip %.2f ms, its parts %.2f" % (whole, parts))
    assert whole <= 1.5 * parts, "%.2f ms against %.2f" % (whole, parts)
    want = torch.linalg.vector_norm(flat, dtype=torch.float64)
    assert abs(float(norm) - float(want)) <= 2.0 ** -23 * float(want)
    got = tg.clip_grads(grads, 1.0, out=outs)
    assert torch.equal(got, norm)
    by = torch.clamp(1.0 / (norm + 1e-6), max=1.0)
    assert torch.equal(out, (flat.float() * by).to(BF))


# ---- the binding without its part in C++ ---------------------------------------------------

@pytest.fixture
def plain_binding(monkeypatch):
    monkeypatch.setattr(ops, "_fast", None)
    monkeypatch.setattr(layers, "_fast", None)
    monkeypatch.setattr(layers, "_entries", {})


def every_operator():
    x, wg, wu, dh = rand(1, 40, 72), rand(2, 56, 72), rand(3, 56, 72), rand(4, 40, 56)
    h, g, u = tg.gemm_glu(x, wg, wu, keep=True)
    odd = tg.gemm_glu(x[:, 1:], wg[:, 1:], wu[:, 1:], act="relu", workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    dx, dwg, dwu = tg.gemm_glu_backward(dh, g, u, x, wg, wu, grad_dtype=F32)
    q, s = tg.int8_quantize(x)
    wq, ws = tg.int8_quantize(wg)
    d, b = tg.gemm_int8(q, s, wq, ws, C=dh, out_dtype=BF), tg.gemm_int8(q, s, wq, ws, C=torch.ones(56, device=DEV))
    norm = tg.grad_norm([dwg, dwu.t(), dx])
    outs = [torch.empty_like(dwg), torch.empty_like(dwu), torch.empty_like(dx)]
    n2 = tg.clip_grads([dwg, dwu, dx], 0.5, out=outs)
    n3 = tg.clip_grads([dwg, dwu.t()], 0.5, given=norm)
    y = tg.rmsnorm(x, rand(5, 72), 1e-5)
    return [h, g, u, odd, dx, dwg, dwu, q, s, wq, ws, d, b, norm, n2, n3, *outs, *y]


def test_operators_through_ctypes(plain_binding, request):
    got = every_operator()
    with pytest.raises(ValueError):
        tg.gemm_glu(rand(1, 4, 8), rand(2, 4, 9), rand(3, 4, 8))
    assert all(isinstance(f, type(layers._load().gemm_glu)) for f in layers._entries.values())
    request.getfixturevalue("monkeypatch").undo()
    for a, b in zip(got, every_operator()):
        assert torch.equal(a, b)


# ---- the range of the gated block's inner gradients ---------------------------------------

def test_glu_backward_range_of_fp16():
    """dg and du as the products' operands, rounded to fp16: 300 x 300 is an infinity, 2^-13 x 1.5 2^-12 rounds to 2^-24
    (du there is 0: act(g) = 2^-14 and dh 2^-13); bf16 holds both."""
    for dtype, big, small in ((FP, float("inf"), 2.0 ** -24), (BF, 300.0 * 300.0, 1.5 * 2.0 ** -25)):
        one = torch.ones(1, 1, device=DEV, dtype=dtype)
        zero = 0 * one
        dx, dwg, _ = tg.gemm_glu_backward(300 * one, one, 300 * one, one, one, zero, act="relu", grad_dtype=F32)
        if dtype == FP:
            assert float(dwg) == big
        else:
            assert abs(float(dwg) / big - 1) <= 2.0 ** -8
        _, dwg, dwu = tg.gemm_glu_backward(2.0 ** -13 * one, 2.0 ** -14 * one, 1.5 * 2.0 ** -12 * one, one, one, zero, act="relu",
                                           grad_dtype=F32)
        assert float(dwg) == small and (float(dwu) == 0 if dtype == FP else float(dwu) == 2.0 ** -27)


def test_clip_over_several_launches_captured():
    """The norm of several launches, added up once, in a graph: replays with new gradients give what the eager call
    gives, in place and into other tensors."""
    n, size = 140, 300001
    flat = torch.zeros(n * size, dtype=BF, device=DEV)
    grads = [flat[i * size:(i + 1) * size] for i in range(n)]
    out, norm, norm2 = torch.zeros_like(flat), torch.zeros((), device=DEV), torch.zeros((), device=DEV)
    outs = [out[i * size:(i + 1) * size] for i in range(n)]
    ws = torch.empty(tg.grad_workspace_bytes(n), dtype=torch.uint8, device=DEV)

    def step():
        tg.clip_grads(grads, 0.75, out=outs, norm=norm, workspace=ws)
        tg.clip_grads(grads, 0.75, norm=norm2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        new = rand(i, n * size, scale=i + 1)
        flat.copy_(new)
        graph.replay()
        again = new.clone()
        want = tg.clip_grads([again[k * size:(k + 1) * size] for k in range(n)], 0.75)
        torch.cuda.synchronize()
        assert torch.equal(norm, want) and torch.equal(norm2, want), "replay %d" % i
        assert torch.equal(flat, again) and torch.equal(out, again), "replay %d" % i
        by = torch.clamp(0.75 / (want + 1e-6), max=1.0)
        assert torch.equal(out, (new.float() * by).to(BF))
        assert abs(float(want) / float(torch.linalg.vector_norm(new, dtype=torch.float64)) - 1) <= 2.0 ** -23
