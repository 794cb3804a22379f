"""Checks of the operators around the block-scaled products on the CPU: the
header's functions are exported, bad arguments are refused before the GPU is
touched (no compute call is made), and the binding refuses host tensors,
types and shapes."""
import os
import re
import subprocess

import pytest
import torch

import tiled_dense_gemm_tile_amd as tg

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "tilegemm_ops.h")
OK, INVALID_SIZE, NULL_POINTER, BAD_LD, MISALIGNED, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 5, 7
F32, BF16, FP16 = 0, 1, 2
P = 0x10000000  # a fake, aligned device address: never dereferenced by these calls
Q = 0x20000000
NAN, INF = float("nan"), float("inf")


def test_header_functions_are_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(\w+)\s*\(", text, flags=re.M)))
    assert names == ["gemm_wgrad_mxfp8", "gemm_wgrad_mxfp8_workspace_bytes", "gemv_mxfp4", "gemv_mxfp4_workspace_bytes",
                     "mxfp8_quantize", "rmsnorm", "rmsnorm_backward", "rmsnorm_backward_workspace_bytes", "rmsnorm_mxfp8"]
    out = subprocess.run(["nm", "-D", "--defined-only", tg.library_path()], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert set(names) <= exported
    # the header is C
    subprocess.run(["gcc", "-fsyntax-only", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-x", "c", HEADER],
                   check=True, capture_output=True)


def quant(rows=4, N=64, X=P, ldx=64, t=BF16, q=Q, ldq=64, sf=Q + 4096, ldsf=2):
    return tg.raw.mxfp8_quantize(rows, N, X, ldx, t, q, ldq, sf, ldsf, None)


def test_quantize_refusals():
    assert quant(rows=-1) == INVALID_SIZE
    assert quant(N=-32) == INVALID_SIZE
    assert quant(rows=1 << 31) == UNSUPPORTED
    assert quant(rows=0, X=None) == OK
    assert quant(N=0) == OK
    assert quant(N=48) == UNSUPPORTED
    assert quant(t=3) == UNSUPPORTED
    assert quant(ldx=63) == BAD_LD
    assert quant(ldq=63) == BAD_LD
    assert quant(ldsf=1) == BAD_LD
    assert quant(X=None) == NULL_POINTER
    assert quant(q=None) == NULL_POINTER
    assert quant(sf=None) == NULL_POINTER
    assert quant(X=P + 1) == MISALIGNED
    assert quant(X=P + 2, t=F32) == MISALIGNED


def norm(rows=4, N=64, X=P, ldx=64, R=P + 4096, ldr=64, t=BF16, W=P + 8192, wt=BF16, eps=1e-5, H=Q, ldh=64,
         Y=Q + 4096, ldy=64, rstd=Q + 8192, mx=False, SF=Q + 12288, ldsf=2):
    if mx:
        return tg.raw.rmsnorm_mxfp8(rows, N, X, ldx, R, ldr, t, W, wt, eps, H, ldh, Y, ldy, SF, ldsf, rstd, None)
    return tg.raw.rmsnorm(rows, N, X, ldx, R, ldr, t, W, wt, eps, H, ldh, Y, ldy, rstd, None)


@pytest.mark.parametrize("mx", [False, True])
def test_norm_refusals(mx):
    assert norm(mx=mx, rows=-1) == INVALID_SIZE
    assert norm(mx=mx, N=-1) == INVALID_SIZE
    assert norm(mx=mx, N=1 << 31) == UNSUPPORTED
    assert norm(mx=mx, rows=0, X=None, W=None) == OK
    assert norm(mx=mx, N=0) == OK
    assert norm(mx=mx, t=7) == UNSUPPORTED
    assert norm(mx=mx, wt=FP16) == UNSUPPORTED
    for eps in (-1e-6, NAN, INF):
        assert norm(mx=mx, eps=eps) == UNSUPPORTED
    for bad in ("ldx", "ldr", "ldh", "ldy"):
        assert norm(mx=mx, **{bad: 63}) == BAD_LD
    for bad in ("X", "W", "Y"):
        assert norm(mx=mx, **{bad: None}) == NULL_POINTER
    for bad in ("X", "R", "H", "W"):
        assert norm(mx=mx, **{bad: P + 1}) == MISALIGNED
    assert norm(mx=mx, rstd=Q + 2) == MISALIGNED
    assert norm(mx=mx, H=Q, Y=Q) == UNSUPPORTED
    assert norm(mx=mx, H=P, ldh=128) == UNSUPPORTED            # in place with another leading dimension
    assert norm(mx=mx, H=P + 4096, ldh=128) == UNSUPPORTED
    if mx:
        assert norm(mx=True, N=40) == UNSUPPORTED
        assert norm(mx=True, ldsf=1) == BAD_LD
        assert norm(mx=True, SF=None) == NULL_POINTER
        assert norm(mx=True, Y=P) == UNSUPPORTED               # codes over the row they come from
    else:
        assert norm(Y=P, ldy=128) == UNSUPPORTED
        assert norm(Y=Q + 4097) == MISALIGNED


def bwd(rows=4, N=64, dY=P, lddy=64, H=P + 4096, ldh=64, t=BF16, W=P + 8192, wt=BF16, rstd=P + 12288, dH=P + 16384,
        lddh=64, dX=Q, lddx=64, dW=Q + 4096, ws=Q + 8192, wb=1 << 20):
    return tg.raw.rmsnorm_backward(rows, N, dY, lddy, H, ldh, t, W, wt, rstd, dH, lddh, dX, lddx, dW, ws, wb, None)


def test_norm_backward_refusals():
    assert bwd(rows=-1) == INVALID_SIZE
    assert bwd(N=-1) == INVALID_SIZE
    assert bwd(N=1 << 31) == UNSUPPORTED
    assert bwd(t=5) == UNSUPPORTED
    assert bwd(wt=FP16) == UNSUPPORTED
    assert bwd(N=0) == OK
    assert bwd(rows=0, dW=None) == OK
    for bad in ("lddy", "ldh", "lddh", "lddx"):
        assert bwd(**{bad: 63}) == BAD_LD
    for bad in ("dY", "H", "W", "rstd", "dX"):
        assert bwd(**{bad: None}) == NULL_POINTER
    for bad in ("dY", "H", "W", "rstd", "dH", "dX", "dW"):
        assert bwd(**{bad: P + 1}) == MISALIGNED
    assert bwd(dX=P + 4096) == UNSUPPORTED                     # over h
    assert bwd(dX=P, lddx=128) == UNSUPPORTED
    assert bwd(dX=P + 16384, lddx=128) == UNSUPPORTED
    assert bwd(ws=None) == WORKSPACE
    assert bwd(wb=tg.rmsnorm_backward_workspace_bytes(4, 64) - 1) == WORKSPACE
    assert bwd(ws=Q + 8192 + 128) == MISALIGNED


def test_norm_backward_workspace_bytes():
    assert tg.rmsnorm_backward_workspace_bytes(0, 64) == 0
    assert tg.rmsnorm_backward_workspace_bytes(-1, 64) == 0
    assert tg.rmsnorm_backward_workspace_bytes(1, 64) == 256
    # bounded however many rows there are
    assert tg.rmsnorm_backward_workspace_bytes(1 << 30, 64) <= 1024 * 64 * 4


def wgrad(M=64, N=64, K=96, A=P, lda=64, B=P + (1 << 20), ldb=64, SF=P + (2 << 20), ldsf=2, C=None, ldc=64, D=Q,
          ldd=64, out=F32, ws=None, wb=0):
    return tg.raw.gemm_wgrad_mxfp8(M, N, K, A, lda, B, ldb, SF, ldsf, C, ldc, D, ldd, out, ws, wb, None)


def test_wgrad_refusals():
    assert wgrad(M=-1) == INVALID_SIZE
    assert wgrad(K=-1) == INVALID_SIZE
    assert wgrad(K=1 << 31) == UNSUPPORTED
    assert wgrad(M=0) == OK
    assert wgrad(N=0, D=None) == OK
    assert wgrad(N=48) == UNSUPPORTED
    assert wgrad(out=FP16) == UNSUPPORTED
    assert wgrad(lda=63) == BAD_LD
    assert wgrad(ldb=32) == BAD_LD
    assert wgrad(ldsf=1) == BAD_LD
    assert wgrad(ldd=63) == BAD_LD
    assert wgrad(C=P, ldc=63) == BAD_LD
    for bad in ("A", "B", "SF", "D"):
        assert wgrad(**{bad: None}) == NULL_POINTER
    assert wgrad(A=P + 1) == MISALIGNED
    assert wgrad(D=Q + 2) == MISALIGNED
    assert wgrad(ws=Q + 64, wb=1 << 20) == MISALIGNED
    assert wgrad(C=Q, ldc=128) == UNSUPPORTED                  # in place with another leading dimension
    assert wgrad(C=Q + 64) == UNSUPPORTED
    assert wgrad(lda=4 << 20) == UNSUPPORTED                   # 8 MiB rows


def test_wgrad_workspace_bytes():
    assert tg.gemm_wgrad_mxfp8_workspace_bytes(0, 64, 64) == 0
    assert tg.gemm_wgrad_mxfp8_workspace_bytes(64, -32, 64) == 0
    assert tg.gemm_wgrad_mxfp8_workspace_bytes(64, 64, 64) == 0
    assert tg.gemm_wgrad_mxfp8_workspace_bytes(8192, 8192, 65536) == 0
    # the partial sums of one round of tiles, however long K is
    assert 0 < tg.gemm_wgrad_mxfp8_workspace_bytes(104, 96, 65536) <= 512 * 128 * 128 * 4
    assert 0 < tg.gemm_wgrad_mxfp8_workspace_bytes(100, 96, 1 << 30) <= 512 * 128 * 128 * 4
    # rows off 16 bytes, a large product: a copy of A too
    assert tg.gemm_wgrad_mxfp8_workspace_bytes(8191, 8192, 65536) == 65536 * 8192 * 2


def gemv(M=2, N=64, K=64, kb=32, X=P, ldx=64, xt=BF16, W=P + (1 << 20), ldw=64, SF=P + (2 << 20), ldsf=2, C=None,
         ldc=64, D=Q, ldd=64, out=F32, ws=None, wb=0):
    return tg.raw.gemv_mxfp4(M, N, K, kb, X, ldx, xt, W, ldw, SF, ldsf, C, ldc, D, ldd, out, ws, wb, None)


def test_gemv_refusals():
    assert gemv(M=-1) == INVALID_SIZE
    assert gemv(N=1 << 31) == UNSUPPORTED
    assert gemv(M=0) == OK
    assert gemv(N=0, D=None) == OK
    assert gemv(xt=F32) == UNSUPPORTED
    assert gemv(out=FP16) == UNSUPPORTED
    assert gemv(K=48) == UNSUPPORTED
    assert gemv(ldw=65) == UNSUPPORTED
    for kb in (0, -32, 16, 40):
        assert gemv(kb=kb) == UNSUPPORTED
    assert gemv(K=192, ldx=192, ldw=192, kb=96) == UNSUPPORTED  # neither a power of two nor one group a row
    assert gemv(ldx=63) == BAD_LD
    assert gemv(ldw=62) == BAD_LD
    assert gemv(ldsf=1) == BAD_LD
    assert gemv(ldd=63) == BAD_LD
    for bad in ("X", "W", "SF", "D"):
        assert gemv(**{bad: None}) == NULL_POINTER
    assert gemv(X=P + 1) == MISALIGNED
    assert gemv(D=Q + 2) == MISALIGNED
    assert gemv(C=Q, ldc=128) == UNSUPPORTED
    assert gemv(ws=Q + 64, wb=1 << 20) == MISALIGNED
    assert gemv(M=(1 << 20) + 1) == UNSUPPORTED


def test_gemv_workspace_bytes():
    assert tg.gemv_mxfp4_workspace_bytes(0, 64, 64) == 0
    assert tg.gemv_mxfp4_workspace_bytes(1, 64, -32) == 0
    assert tg.gemv_mxfp4_workspace_bytes(1, 14336, 4096) == 0
    b = tg.gemv_mxfp4_workspace_bytes(16, 4096, 14336)
    assert b > 0 and b % (16 * 4096 * 4) == 0


def test_binding_refuses_host_tensors_and_types():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tg.mxfp8_quantize(x)
    with pytest.raises(ValueError):
        tg.rmsnorm(x, w, 1e-5)
    with pytest.raises(ValueError):
        tg.rmsnorm_mxfp8(x, w, 1e-5)
    with pytest.raises(ValueError):
        tg.rmsnorm_backward(x, x, w, torch.zeros(4))
    with pytest.raises(ValueError):
        tg.gemm_wgrad_mxfp8(x, torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError):
        tg.gemv_mxfp4(x, torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8))
    with pytest.raises(TypeError):
        tg.mxfp8_quantize(x.int())
    with pytest.raises(TypeError):
        tg.gemv_mxfp4(x.float(), torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8))
    with pytest.raises(TypeError):
        tg.gemm_wgrad_mxfp8(x.half(), torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))


def test_limits_of_row_lengths():
    n = 1 << 28
    assert quant(N=n, ldx=n, ldq=n, ldsf=n // 32) == UNSUPPORTED
    for mx in (False, True):
        assert norm(mx=mx, N=n, ldx=n, ldr=n, ldh=n, ldy=n, ldsf=n // 32) == UNSUPPORTED
    assert bwd(N=n, lddy=n, ldh=n, lddh=n, lddx=n) == UNSUPPORTED
    assert tg.rmsnorm_backward_workspace_bytes(4, n) == 0


def test_outputs_over_each_other_are_refused():
    assert quant(q=P) == UNSUPPORTED
    assert quant(sf=P) == UNSUPPORTED
    assert quant(q=Q, sf=Q) == UNSUPPORTED
    assert norm(mx=True, Y=Q + 4096, SF=Q + 4096) == UNSUPPORTED


def test_gemv_workspace_is_bounded():
    """However many rows of X there are: 64 MiB, or 32 rows' partial sums."""
    for m, n, k in ((1 << 20, 14336, 16384), (4096, 4096, 14336), (1 << 20, 64, 1 << 20)):
        splits = -(-k // 1024)
        assert 0 < tg.gemv_mxfp4_workspace_bytes(m, n, k) <= max(64 << 20, splits * 32 * n * 4)


@pytest.mark.parametrize("out,n", [(F32, 1 << 21), (1, 1 << 22)], ids=["f32", "bf16"])
def test_gemv_refuses_more_columns_than_a_row_of_d_holds(out, n):
    """N is bounded by ldd's limit of 8 MiB, far below what one launch counts (2^32 threads, 512 for 16 columns)."""
    assert n // 16 * 512 < 1 << 32
    for big in (n, 1 << 27, (1 << 31) - 1):
        assert gemv(M=1, N=big, K=32, ldx=32, ldw=32, ldsf=1, ldd=big, out=out) == UNSUPPORTED
        assert gemv(M=1, N=big, K=32, ldx=32, ldw=32, ldsf=1, ldd=n - 1, out=out) == BAD_LD
