"""Checks of the feed-forward layer's operators on the CPU: the header's
functions are exported, bad arguments are refused before the GPU is touched
(no compute call is made), and the binding refuses host tensors, types and
shapes."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import tiled_dense_gemm_tile_amd as tg

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "tilegemm_layers.h")
OK, INVALID_SIZE, NULL_POINTER, BAD_LD, MISALIGNED, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 5, 7
F32, BF16, FP16 = 0, 1, 2
MB = 1 << 20
P = 0x10000000  # fake, aligned device addresses: never dereferenced by these calls
Q = 0x20000000
NAN, INF = float("nan"), float("inf")


def test_header_functions_are_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(\w+)\s*\(", text, flags=re.M)))
    assert names == ["gemm_glu", "gemm_glu_backward", "gemm_glu_backward_workspace_bytes", "gemm_glu_workspace_bytes", "gemm_int8",
                     "gemm_int8_workspace_bytes", "grad_clip", "grad_norm", "grad_workspace_bytes", "int8_quantize"]
    out = subprocess.run(["nm", "-D", "--defined-only", tg.library_path()], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert set(names) <= exported
    subprocess.run(["gcc", "-fsyntax-only", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-x", "c", HEADER],
                   check=True, capture_output=True)


def glu(M=4, F=64, K=32, X=P, ldx=32, Wg=P + MB, ldwg=32, Wu=P + 2 * MB, ldwu=32, t=BF16, act=0, H=Q, ldh=64,
        G=Q + MB, ldg=64, U=Q + 2 * MB, ldu=64, ws=None, wb=0):
    return tg.raw.gemm_glu(M, F, K, X, ldx, Wg, ldwg, Wu, ldwu, t, act, H, ldh, G, ldg, U, ldu, ws, wb, None)


def test_glu_refusals():
    for bad in ("M", "F", "K"):
        assert glu(**{bad: -1}) == INVALID_SIZE
        assert glu(**{bad: 1 << 31}) == UNSUPPORTED
    assert glu(M=0, X=None) == OK
    assert glu(F=0, H=None) == OK
    for t in (F32, 3, -1):
        assert glu(t=t) == UNSUPPORTED
    for act in (-1, 4):
        assert glu(act=act) == UNSUPPORTED
    for bad in ("ldx", "ldwg", "ldwu"):
        assert glu(**{bad: 31}) == BAD_LD
        assert glu(**{bad: 4 * MB}) == UNSUPPORTED             # 8 MiB rows
    for bad in ("ldh", "ldg", "ldu"):
        assert glu(**{bad: 63}) == BAD_LD
        assert glu(**{bad: 4 * MB}) == UNSUPPORTED
    for bad in ("X", "Wg", "Wu", "H"):
        assert glu(**{bad: None}) == NULL_POINTER
    for bad in ("X", "Wg", "Wu", "H", "G", "U"):
        assert glu(**{bad: P + 8 * MB + 1}) == MISALIGNED
    for bad in ("H", "G", "U"):
        assert glu(**{bad: P}) == UNSUPPORTED                  # over X
        assert glu(**{bad: P + MB + 64}) == UNSUPPORTED        # over Wg
    assert glu(G=Q) == UNSUPPORTED
    assert glu(U=Q + MB) == UNSUPPORTED
    assert glu(ws=Q + 4 * MB + 128, wb=MB) == MISALIGNED


def test_workspace_bytes_of_copies():
    """Large grids alone, and copies that few results would read are left out: rows of an odd multiple of 256 bytes."""
    for f in (tg.gemm_glu_workspace_bytes, tg.gemm_int8_workspace_bytes):
        for none in ((0, 4096, 4096), (4096, -1, 4096), (4096, 4096, 0), (32, 4096, 4095), (1 << 31, 4096, 64), (256, 1 << 20, 65)):
            assert f(*none) == 0
    assert tg.gemm_glu_workspace_bytes(4096, 4095, 1001) == (4096 + 2 * 4095) * 2304
    assert tg.gemm_int8_workspace_bytes(4096, 4095, 1001) == (4096 + 4095) * 1280


def bwd(M=4, F=64, K=32, dH=P, lddh=64, G=P + MB, ldg=64, U=P + 2 * MB, ldu=64, X=P + 3 * MB, ldx=32, Wg=P + 4 * MB,
        ldwg=32, Wu=P + 5 * MB, ldwu=32, t=BF16, act=0, dX=Q, lddx=32, Cg=None, ldcg=32, Cu=None, ldcu=32, dWg=Q + MB,
        lddwg=32, dWu=Q + 2 * MB, lddwu=32, gt=BF16, ws=Q + 3 * MB, wb=MB):
    return tg.raw.gemm_glu_backward(M, F, K, dH, lddh, G, ldg, U, ldu, X, ldx, Wg, ldwg, Wu, ldwu, t, act, dX, lddx, Cg,
                                    ldcg, Cu, ldcu, dWg, lddwg, dWu, lddwu, gt, ws, wb, None)


def test_glu_backward_refusals():
    for bad in ("M", "F", "K"):
        assert bwd(**{bad: -1}) == INVALID_SIZE
    assert bwd(M=1 << 21) == UNSUPPORTED
    assert bwd(F=1 << 20) == UNSUPPORTED
    assert bwd(K=1 << 31) == UNSUPPORTED
    assert bwd(K=0, dH=None) == OK
    assert bwd(dX=None, dWg=None, dWu=None, dH=None) == OK     # nothing is wanted
    assert bwd(M=0, dWg=None, dWu=None) == OK
    assert bwd(F=0, dX=None) == OK
    assert bwd(t=F32) == UNSUPPORTED
    assert bwd(act=7) == UNSUPPORTED
    assert bwd(gt=FP16) == UNSUPPORTED
    for bad in ("lddh", "ldg", "ldu"):
        assert bwd(**{bad: 63}) == BAD_LD
        assert bwd(**{bad: 4 * MB}) == UNSUPPORTED
    for bad in ("ldx", "ldwg", "ldwu", "lddx", "lddwg", "lddwu"):
        assert bwd(**{bad: 31}) == BAD_LD
        assert bwd(**{bad: 4 * MB}) == UNSUPPORTED
    c = dict(Cg=P + 6 * MB, Cu=P + 7 * MB)
    for bad in ("ldcg", "ldcu"):
        assert bwd(**c, **{bad: 31}) == BAD_LD
        assert bwd(**c, **{bad: 4 * MB}) == UNSUPPORTED
    for bad in ("dH", "G", "U", "X", "Wg", "Wu", "dWg", "dWu"):
        assert bwd(**{bad: None}) == NULL_POINTER
    assert bwd(Cg=P + 6 * MB) == NULL_POINTER                  # one of both
    assert bwd(**c, dWg=None, dWu=None) == NULL_POINTER
    for bad in ("dH", "G", "U", "X", "Wg", "Wu", "dX", "dWg", "dWu"):
        assert bwd(**{bad: P + 9 * MB + 1}) == MISALIGNED
    assert bwd(gt=F32, dWg=Q + MB + 2) == MISALIGNED
    for bad in ("dX", "dWg", "dWu"):
        for src in range(6):
            assert bwd(**{bad: P + src * MB}) == UNSUPPORTED
    assert bwd(dWu=Q + MB) == UNSUPPORTED                      # both gradients in one place
    assert bwd(dX=Q + MB) == UNSUPPORTED
    assert bwd(Cg=Q + MB, Cu=Q + 2 * MB, ldcg=64) == UNSUPPORTED   # in place with another leading dimension
    assert bwd(Cg=Q + MB + 64, Cu=P + 7 * MB) == UNSUPPORTED   # partly over its result
    assert bwd(Cg=Q + 2 * MB, Cu=Q + MB) == UNSUPPORTED        # the other's result
    assert bwd(ws=None) == WORKSPACE
    assert bwd(wb=tg.gemm_glu_backward_workspace_bytes(4, 64, 32) - 1) == WORKSPACE
    assert bwd(ws=Q + 3 * MB + 128) == MISALIGNED


def test_glu_backward_workspace_bytes():
    assert tg.gemm_glu_backward_workspace_bytes(4, 0, 32) == 0
    assert tg.gemm_glu_backward_workspace_bytes(-1, 64, 32) == 0
    assert tg.gemm_glu_backward_workspace_bytes(1 << 21, 64, 32) == 0
    # dg | du, both transposed, X and the weights transposed: tiles of 64, rows of an odd multiple of 256 bytes
    assert tg.gemm_glu_backward_workspace_bytes(100, 70, 32) == 2 * (100 * 384 + 256 * 128 + 32 * 128 + 32 * 384)


def quant(rows=4, N=64, X=P, ldx=64, t=BF16, q=Q, ldq=64, s=Q + MB):
    return tg.raw.int8_quantize(rows, N, X, ldx, t, q, ldq, s, None)


def test_quantize_refusals():
    assert quant(rows=-1) == INVALID_SIZE
    assert quant(N=-1) == INVALID_SIZE
    assert quant(rows=1 << 31) == UNSUPPORTED
    assert quant(N=1 << 28, ldx=1 << 28, ldq=1 << 28) == UNSUPPORTED
    assert quant(rows=0, X=None) == OK
    assert quant(t=3) == UNSUPPORTED
    assert quant(ldx=63) == BAD_LD
    assert quant(ldq=63) == BAD_LD
    for bad in ("X", "q", "s"):
        assert quant(**{bad: None}) == NULL_POINTER
    assert quant(X=P + 1) == MISALIGNED
    assert quant(s=Q + MB + 2) == MISALIGNED
    assert quant(q=P) == UNSUPPORTED
    assert quant(s=P + 4) == UNSUPPORTED
    assert quant(s=Q + 8) == UNSUPPORTED


def int8(M=4, N=64, K=32, A=P, lda=32, SA=P + MB, B=P + 2 * MB, ldb=32, SB=P + 3 * MB, C=None, ldc=64, D=Q, ldd=64,
         out=F32, ws=None, wb=0):
    return tg.raw.gemm_int8(M, N, K, A, lda, SA, B, ldb, SB, C, ldc, D, ldd, out, ws, wb, None)


def test_int8_refusals():
    for bad in ("M", "N", "K"):
        assert int8(**{bad: -1}) == INVALID_SIZE
    assert int8(M=1 << 31) == UNSUPPORTED
    assert int8(K=1 << 17, lda=1 << 17, ldb=1 << 17) == UNSUPPORTED
    assert int8(M=0, A=None) == OK
    assert int8(N=0, D=None) == OK
    assert int8(out=3) == UNSUPPORTED
    assert int8(lda=31) == BAD_LD
    assert int8(ldb=31) == BAD_LD
    assert int8(ldd=63) == BAD_LD
    assert int8(C=P + 4 * MB, ldc=63) == BAD_LD
    assert int8(C=P + 4 * MB, ldc=1) == BAD_LD
    for bad in ("A", "B", "SA", "SB", "D"):
        assert int8(**{bad: None}) == NULL_POINTER
    for bad in ("SA", "SB", "D", "C"):
        assert int8(**{bad: P + 5 * MB + 2}) == MISALIGNED
    assert int8(lda=8 * MB) == UNSUPPORTED
    assert int8(ws=Q + 4 * MB + 8, wb=MB) == MISALIGNED
    assert int8(ldd=2 * MB) == UNSUPPORTED
    assert int8(C=Q, ldc=128) == UNSUPPORTED                   # in place with another leading dimension
    assert int8(C=Q + 64) == UNSUPPORTED
    assert int8(C=Q + 64, ldc=0) == UNSUPPORTED                # a bias inside the result
    for src in range(4):
        assert int8(D=P + src * MB) == UNSUPPORTED


def grads(at=(P, P + MB), sizes=(10, 20), types=(BF16, F32), out=None, top=1.0, given=None, norm=Q, ws=Q + MB, wb=MB,
          clip=True, n=None):
    n = len(at) if n is None else n
    a = (ctypes.c_void_p * len(at))(*at)
    o = (ctypes.c_void_p * len(at))(*(at if out is None else out))
    s, t = (ctypes.c_int64 * len(sizes))(*sizes), (ctypes.c_int * len(types))(*types)
    if clip:
        return tg.raw.grad_clip(n, a, o, s, t, top, given, norm, ws, wb, None)
    return tg.raw.grad_norm(n, a, s, t, norm, ws, wb, None)


@pytest.mark.parametrize("clip", [True, False])
def test_gradient_refusals(clip):
    assert grads(clip=clip, n=-1) == INVALID_SIZE
    assert grads(clip=clip, n=1 << 20) == UNSUPPORTED
    assert grads(clip=clip, sizes=(10, -1)) == INVALID_SIZE
    assert grads(clip=clip, sizes=(10, 1 << 40)) == UNSUPPORTED
    assert grads(clip=clip, sizes=((1 << 39), (1 << 39))) == UNSUPPORTED
    assert grads(clip=clip, types=(BF16, 3)) == UNSUPPORTED
    assert grads(clip=clip, at=(P, None)) == NULL_POINTER
    assert grads(clip=clip, norm=None) == NULL_POINTER
    assert grads(clip=clip, at=(P + 1, P + MB)) == MISALIGNED
    assert grads(clip=clip, at=(P, P + 2)) == MISALIGNED       # fp32
    assert grads(clip=clip, norm=Q + 1) == MISALIGNED
    assert grads(clip=clip, ws=None) == WORKSPACE
    assert grads(clip=clip, wb=tg.grad_workspace_bytes(2) - 1) == WORKSPACE
    assert grads(clip=clip, ws=Q + MB + 8) == MISALIGNED


def test_clip_refusals():
    assert grads(top=-1.0) == UNSUPPORTED
    assert grads(top=NAN) == UNSUPPORTED
    assert grads(out=(P, None)) == NULL_POINTER
    assert grads(out=(P, P + MB + 1)) == MISALIGNED
    assert grads(given=Q + 1) == MISALIGNED


def test_gradient_workspace_bytes():
    assert tg.grad_workspace_bytes(-1) == 0
    assert tg.grad_workspace_bytes(1 << 20) == 0
    assert 0 < tg.grad_workspace_bytes(0) <= tg.grad_workspace_bytes(1) <= tg.grad_workspace_bytes(1000) <= 1 << 18


def test_binding_refuses_host_tensors_and_types():
    x, w, q = torch.zeros(4, 64).bfloat16(), torch.zeros(8, 64).bfloat16(), torch.zeros(4, 64, dtype=torch.int8)
    h, s = torch.zeros(4, 8).bfloat16(), torch.zeros(4)
    for call in (lambda: tg.gemm_glu(x, w, w), lambda: tg.gemm_glu_backward(h, h, h, x, w, w), lambda: tg.int8_quantize(x),
                 lambda: tg.gemm_int8(q, s, q, s), lambda: tg.grad_norm([x]), lambda: tg.clip_grads([x], 1.0),
                 lambda: tg.grad_norm([])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: tg.gemm_glu(x.float(), w.float(), w.float()), lambda: tg.gemm_glu(x[0], w, w),
                 lambda: tg.gemm_glu_backward(h, h, h, x.float(), w, w), lambda: tg.int8_quantize(x.int()),
                 lambda: tg.gemm_int8(x, s, q, s)):
        with pytest.raises(TypeError):
            call()


def test_checks_in_cpp_say_what_python_says():
    """The binding's checks in C++ against their Python form, over every way a matrix or a vector can be wrong."""
    fast = pytest.importorskip("tiled_dense_gemm_tile_amd._tensors")
    from tiled_dense_gemm_tile_amd import ops
    bf, f32 = (torch.bfloat16,), (torch.float32, torch.bfloat16)
    m = torch.zeros(6, 10).bfloat16()
    cases = [(m, (6, 10), bf), (m, (6, 10), f32), (m, (6, 10), (torch.float16,)), (m, (5, 10), bf), (m[:, :4], (6, 4), bf),
             (m.t(), (10, 6), bf), (m[::2], (3, 10), bf), (m[:, ::2], (6, 5), bf), (m[:, :1], (6, 1), bf), (m[:1], (1, 10), bf),
             (m[2:3, :4], (1, 4), bf), (m[:0], (0, 10), bf), (m[0], (1, 10), bf), (m[:, :0], (6, 0), bf),
             (m.as_strided((1, 10), (1 << 22, 1)), (1, 10), bf), (m.as_strided((1, 10), (3, 1)), (1, 10), bf)]
    slow, ops._fast = ops._fast, None
    try:
        for t, shape, types in cases:
            for dev in (-1, 0):
                try:
                    want = ops._matrix("t", t, shape, types, dev)
                except (TypeError, ValueError):
                    want = None
                assert fast.matrix(t, shape, types, dev) == want, (t.shape, t.stride(), shape, types, dev)
        v = torch.zeros(12)
        for t, n, types in ((v, 12, f32), (v, 11, f32), (v, 12, bf), (v[::2], 6, f32), (v[:1], 1, f32), (v[::12], 1, f32), (m, 6, f32)):
            for dev in (-1, 0):
                try:
                    want = ops._vector("t", t, n, types, dev)
                except (TypeError, ValueError):
                    want = None
                assert fast.vector(t, n, types, dev) == want
    finally:
        ops._fast = slow
    assert fast.matrix(None, (1, 1), bf, -1) is None and fast.matrix(m.to_sparse(), (6, 10), bf, -1) is None
    # lists on the host, of other types, or empty are left to Python
    assert fast.gradients([]) is None and fast.gradients([m]) is None and fast.gradients([1]) is None


def test_calls_in_cpp_refuse_wrong_counts():
    fast = pytest.importorskip("tiled_dense_gemm_tile_amd._tensors")
    from tiled_dense_gemm_tile_amd import layers
    f = layers._entry("gemm_int8")
    assert f is fast.gemm_int8
    with pytest.raises(TypeError):
        f(1, 2, 3)
    with pytest.raises(TypeError):
        f(*["x"] * 17)
    assert f(-1, 4, 4, 1, 64, 1, 1, 64, 1, None, 0, 1, 64, 0, None, 0, None) == INVALID_SIZE


def test_shared_memory_is_refused():
    """Matrices that share elements; those of one leading dimension that lie next to each other row by row do not."""
    assert glu(G=Q + 64) == UNSUPPORTED                        # rows of 128 bytes, half a row on
    assert glu(ldh=128, ldg=128, G=Q + 126) == UNSUPPORTED     # one element too near
    assert glu(ldh=128, ldg=130, G=Q + 128) == UNSUPPORTED     # rows that drift apart
    assert glu(ldu=128, ldg=128, U=Q + MB + 130) == UNSUPPORTED    # the last element is the next row's first
    assert bwd(dWu=Q + MB + 32) == UNSUPPORTED
    assert bwd(lddwg=64, lddwu=64, dWu=Q + MB + 62) == UNSUPPORTED
    assert bwd(dX=Q + MB + 64) == UNSUPPORTED
    assert bwd(Cg=P + 6 * MB, Cu=Q + MB + 64) == UNSUPPORTED   # Cu in the other's result
    for at in (P, P + 3 * MB, P + 5 * MB, Q, Q + 2 * MB):      # the workspace over an operand, a result
        assert bwd(ws=at) == UNSUPPORTED
    assert int8(ldc=128, ldd=128, C=Q + 252) == UNSUPPORTED
    big = dict(M=4096, N=4095, K=1001, lda=1001, ldb=1001, ldd=4095, SA=P + 32 * MB, SB=P + 33 * MB, B=P + 16 * MB)
    need = tg.gemm_int8_workspace_bytes(4096, 4095, 1001)
    for at in (P, P + 16 * MB, P + 32 * MB, Q, Q + 63 * MB):   # where operands are copied
        assert int8(**big, ws=at, wb=need) == UNSUPPORTED
    big = dict(M=4096, F=4095, K=1001, ldx=1001, ldwg=1001, ldwu=1001, ldh=4095, G=None, U=None, Wg=P + 16 * MB, Wu=P + 32 * MB)
    need = tg.gemm_glu_workspace_bytes(4096, 4095, 1001)
    for at in (P, P + 16 * MB, P + 32 * MB, Q, Q + 31 * MB):
        assert glu(**big, ws=at, wb=need) == UNSUPPORTED


def test_gradients_that_share_memory_are_refused():
    two = dict(sizes=(10, 20), types=(BF16, F32))
    assert grads(at=(P + 4, P), **two) == UNSUPPORTED          # the first inside the second
    assert grads(at=(P, P + 16), **two) == UNSUPPORTED         # the second in the first's last elements
    assert grads(out=(Q + 2 * MB, Q + 2 * MB + 16), **two) == UNSUPPORTED
    assert grads(out=(P + MB, Q + 2 * MB), **two) == UNSUPPORTED   # a result over the other's gradient
    assert grads(out=(P + 2, P + MB), **two) == UNSUPPORTED    # over its own, shifted
    assert grads(norm=P + MB + 76) == UNSUPPORTED
    assert grads(given=P + 8, norm=None) == UNSUPPORTED
    assert grads(at=(P, Q + MB + 64)) == UNSUPPORTED           # in the workspace
    n = 1000                                                   # many: one overlap at a time, anywhere
    for k in (0, 1, 500, 998):
        at = [P + 4096 * ((7 * i) % n) for i in range(n)]
        at[k + 1] = at[k] + 16
        assert grads(at=at, sizes=[8] * n, types=[F32] * n) == UNSUPPORTED


def test_sizes_that_no_grid_holds():
    assert glu(M=1 << 27) == UNSUPPORTED
    assert glu(F=1 << 27, ldh=1 << 27) == UNSUPPORTED
    assert int8(M=1 << 27) == UNSUPPORTED
    assert int8(N=1 << 27, ldd=1 << 27) == UNSUPPORTED
    assert tg.gemm_glu_workspace_bytes(1 << 27, 4096, 65) == 0
    # copies' rows: 2 K bytes rounded up to an odd multiple of 256, the largest of which below 8 MiB is 8 MiB - 256
    assert tg.gemm_glu_workspace_bytes(4096, 4095, 4 * MB - 127) == 0
    assert tg.gemm_glu_workspace_bytes(4096, 4095, 4 * MB - 129) == (4096 + 2 * 4095) * (8 * MB - 256)
