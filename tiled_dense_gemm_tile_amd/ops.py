"""Binding of ``include/tilegemm_ops.h``: the operators around the
block-scaled products.

Training: ``rmsnorm_mxfp8`` (or ``mxfp8_quantize``) makes the A and SFA of
``gemm_mxfp8``; the backward pass takes the weight gradient from that same
8-bit operand (``gemm_wgrad_mxfp8``), the input gradient from ``gemm_bf16``
and the norm's from ``rmsnorm_backward``.  Serving: ``rmsnorm`` and
``gemv_mxfp4`` for a few tokens.

Tensors are 2-D with a last stride of 1; the first stride is the leading
dimension.  Outputs not given are allocated.  Calls are enqueued on torch's
current stream of the tensors' GPU.
"""
from __future__ import annotations

import torch

from . import OUT_BF16, OUT_F32, _check, _ld, _load, _on_device

_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_E4M3 = (torch.float8_e4m3fn, torch.uint8)
_E8M0 = (torch.float8_e8m0fnu, torch.uint8)


def _run(name, dev, *args):
    """The C call on torch's current stream of ``dev``, with ``dev`` current
    (a NULL stream means the current device's)."""
    f = getattr(_load(), name)
    stream = torch.cuda.current_stream(dev).cuda_stream
    if torch.cuda.current_device() == dev.index:
        _check(f(*args, stream))
    else:
        with torch.cuda.device(dev):
            _check(f(*args, stream))


def _matrix(name, t, rows, cols, dtypes):
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s" % (name, " or ".join(str(d) for d in dtypes)))
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError("%s must be (%d, %d)" % (name, rows, cols))
    return t


def _vector(name, t, n, dtypes):
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s" % (name, " or ".join(str(d) for d in dtypes)))
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError("%s must be a contiguous vector of %d" % (name, n))
    return t


def _ptr_ld(t, cols):
    return (None, 0) if t is None else (t.data_ptr(), _ld(t, cols))


def _rows(X):
    if X.dim() != 2 or X.dtype not in _TYPES:
        raise TypeError("X must be a 2-D float32, bfloat16 or float16 tensor")
    _on_device(X, X=X)
    return X.shape[0], X.shape[1], X.dtype


def _scaled_out(X, rows, N, Q, SF):
    if N % 32:
        raise ValueError("block-scaled rows hold a multiple of 32 elements")
    if Q is None:
        Q = torch.empty((rows, N), dtype=torch.float8_e4m3fn, device=X.device)
    if SF is None:
        SF = torch.empty((rows, N // 32), dtype=torch.float8_e8m0fnu, device=X.device)
    return _matrix("Q", Q, rows, N, _E4M3), _matrix("SF", SF, rows, N // 32, _E8M0)


def mxfp8_quantize(X, Q=None, SF=None):
    """X (rows, N) as block-scaled rows: e4m3 codes Q (rows, N) and e8m0
    scales SF (rows, N/32), as :func:`gemm_mxfp8` takes an operand.  N must
    be a multiple of 32.  The scale of a block is the least power of two that
    clips none of its elements.  Returns (Q, SF)."""
    rows, N, dtype = _rows(X)
    Q, SF = _scaled_out(X, rows, N, Q, SF)
    _on_device(X, Q=Q, SF=SF)
    _run("mxfp8_quantize", X.device, rows, N, X.data_ptr(), _ld(X, N), _TYPES[dtype], Q.data_ptr(), _ld(Q, N),
         SF.data_ptr(), _ld(SF, N // 32))
    return Q, SF


def _norm_args(X, W, residual, H, rstd):
    rows, N, dtype = _rows(X)
    _vector("W", W, N, (dtype, torch.float32))
    if residual is not None:
        _matrix("residual", residual, rows, N, (dtype,))
        if H is None:
            H = torch.empty((rows, N), dtype=dtype, device=X.device)
    if H is not None:
        _matrix("H", H, rows, N, (dtype,))
    if rstd is None:
        rstd = torch.empty(rows, dtype=torch.float32, device=X.device)
    _vector("rstd", rstd, rows, (torch.float32,))
    return rows, N, dtype, H, rstd


def rmsnorm(X, W, eps, residual=None, Y=None, H=None, rstd=None):
    """Root-mean-square norm of each row of H = X + residual (rounded to X's
    type; X itself without a residual): Y = H * W * rstd, rstd = 1 /
    sqrt(mean(H^2) + eps).  W (N,) of X's type or float32.  H may be given as
    X or the residual (in place), and so may Y unless H is the same.
    Returns (Y, H, rstd), H being X when there is no residual and no H."""
    rows, N, dtype, H, rstd = _norm_args(X, W, residual, H, rstd)
    if Y is None:
        Y = torch.empty((rows, N), dtype=dtype, device=X.device)
    _matrix("Y", Y, rows, N, (dtype,))
    _on_device(X, W=W, residual=residual, H=H, Y=Y, rstd=rstd)
    rp, ldr = _ptr_ld(residual, N)
    hp, ldh = _ptr_ld(H, N)
    _run("rmsnorm", X.device, rows, N, X.data_ptr(), _ld(X, N), rp, ldr, _TYPES[dtype], W.data_ptr(),
         _TYPES[W.dtype], float(eps), hp, ldh, Y.data_ptr(), _ld(Y, N), rstd.data_ptr())
    return Y, X if H is None else H, rstd


def rmsnorm_mxfp8(X, W, eps, residual=None, Q=None, SF=None, H=None, rstd=None):
    """:func:`rmsnorm` with the result as block-scaled rows (see
    :func:`mxfp8_quantize`): the operand of :func:`gemm_mxfp8` and the 8-bit
    copy that :func:`gemm_wgrad_mxfp8` reads in the backward pass.  Returns
    (Q, SF, H, rstd)."""
    rows, N, dtype, H, rstd = _norm_args(X, W, residual, H, rstd)
    Q, SF = _scaled_out(X, rows, N, Q, SF)
    _on_device(X, W=W, residual=residual, H=H, Q=Q, SF=SF, rstd=rstd)
    rp, ldr = _ptr_ld(residual, N)
    hp, ldh = _ptr_ld(H, N)
    _run("rmsnorm_mxfp8", X.device, rows, N, X.data_ptr(), _ld(X, N), rp, ldr, _TYPES[dtype], W.data_ptr(),
         _TYPES[W.dtype], float(eps), hp, ldh, Q.data_ptr(), _ld(Q, N), SF.data_ptr(), _ld(SF, N // 32),
         rstd.data_ptr())
    return Q, SF, X if H is None else H, rstd


def rmsnorm_backward_workspace_bytes(rows: int, N: int) -> int:
    """Workspace bytes :func:`rmsnorm_backward` needs for dW."""
    return int(_load().rmsnorm_backward_workspace_bytes(rows, N))


def rmsnorm_backward(dY, H, W, rstd, dH=None, dX=None, dW=None, workspace=None, weight_grad=True):
    """Gradients of :func:`rmsnorm` / :func:`rmsnorm_mxfp8` from the gradient
    dY of its result: dX (dY's type; the gradient of X and of the residual
    alike) and dW (float32; None with ``weight_grad=False``).  H and rstd as
    the forward call returned them; ``dH``: the gradient that reaches H from
    elsewhere, added to dX.  dX may be given as dY or dH (in place).
    ``workspace``: a device byte tensor of at least
    :func:`rmsnorm_backward_workspace_bytes` bytes, 256-byte aligned
    (allocated per call when not given).  Returns (dX, dW)."""
    rows, N, dtype = _rows(dY)
    _matrix("H", H, rows, N, (dtype,))
    _vector("W", W, N, (dtype, torch.float32))
    _vector("rstd", rstd, rows, (torch.float32,))
    if dH is not None:
        _matrix("dH", dH, rows, N, (dtype,))
    if dX is None:
        dX = torch.empty((rows, N), dtype=dtype, device=dY.device)
    _matrix("dX", dX, rows, N, (dtype,))
    wp, wb = None, 0
    if weight_grad:
        if dW is None:
            dW = torch.empty(N, dtype=torch.float32, device=dY.device)
        _vector("dW", dW, N, (torch.float32,))
        if workspace is None:
            workspace = torch.empty(rmsnorm_backward_workspace_bytes(rows, N), dtype=torch.uint8, device=dY.device)
        wp, wb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif dW is not None:
        raise ValueError("dW given with weight_grad=False")
    _on_device(dY, H=H, W=W, rstd=rstd, dH=dH, dX=dX, dW=dW, workspace=workspace)
    hp, ldh = _ptr_ld(dH, N)
    _run("rmsnorm_backward", dY.device, rows, N, dY.data_ptr(), _ld(dY, N), H.data_ptr(), _ld(H, N), _TYPES[dtype],
         W.data_ptr(), _TYPES[W.dtype], rstd.data_ptr(), hp, ldh, dX.data_ptr(), _ld(dX, N),
         None if dW is None else dW.data_ptr(), wp, wb)
    return dX, dW


def _product_out(ref, M, N, C, D, out_dtype):
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out_dtype must be float32 or bfloat16")
    if D is None:
        D = torch.empty((M, N), dtype=out_dtype, device=ref.device)
    _matrix("D", D, M, N, (out_dtype,))
    if C is not None:
        _matrix("C", C, M, N, (out_dtype,))
    return D, OUT_BF16 if out_dtype == torch.bfloat16 else OUT_F32


def gemm_wgrad_mxfp8_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace bytes with which :func:`gemm_wgrad_mxfp8` may cut K (0: it
    would not)."""
    return int(_load().gemm_wgrad_mxfp8_workspace_bytes(M, N, K))


def gemm_wgrad_mxfp8(dY, Q, SF, C=None, out_dtype=None, D=None, workspace=None):
    """Weight gradient from an 8-bit activation: D (M, N) = dY^T @ X + C, dY
    (K tokens, M) bfloat16 and X (K, N) given as block-scaled rows Q, SF
    (:func:`mxfp8_quantize`, :func:`rmsnorm_mxfp8`).  ``out_dtype`` float32
    (default) or bfloat16, C of that type; C may be D (gradient
    accumulation).  ``workspace``: a device byte tensor, 256-byte aligned, of
    :func:`gemm_wgrad_mxfp8_workspace_bytes` bytes (allocated per call when
    not given; a smaller one runs without cutting K)."""
    if dY.dtype != torch.bfloat16 or dY.dim() != 2:
        raise TypeError("dY must be a 2-D bfloat16 tensor")
    _on_device(dY, dY=dY)
    K, M = dY.shape
    if Q.dim() != 2 or Q.shape[1] % 32:
        raise ValueError("Q must be (K, N) with N a multiple of 32")
    N = Q.shape[1]
    _matrix("Q", Q, K, N, _E4M3)
    _matrix("SF", SF, K, N // 32, _E8M0)
    D, out = _product_out(dY, M, N, C, D, out_dtype)
    if workspace is None:
        need = gemm_wgrad_mxfp8_workspace_bytes(M, N, K)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dY.device)
    _on_device(dY, Q=Q, SF=SF, C=C, D=D, workspace=workspace)
    wp, wb = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    cp, ldc = _ptr_ld(C, N)
    _run("gemm_wgrad_mxfp8", dY.device, M, N, K, dY.data_ptr(), _ld(dY, M), Q.data_ptr(), _ld(Q, N), SF.data_ptr(),
         _ld(SF, N // 32), cp, ldc, D.data_ptr(), _ld(D, N), out, wp, wb)
    return D


def gemv_mxfp4(X, W, SFW, kblock=32, C=None, out_dtype=None, D=None):
    """A few rows times 4-bit weights: D (M, N) = X @ W^T + C, X (M, K)
    bfloat16 or float16, W (N, K/2) bytes of two e2m1 codes and SFW (N,
    ceil(K / kblock)) e8m0 codes, as :func:`gemm_mxfp4` and
    :func:`gemm_mx_kblock` take B and SFB.  X is not quantised.  Made for up
    to 16 rows, right for any number.  ``out_dtype`` float32 (default) or
    bfloat16; C of that type may be D."""
    if X.dtype not in (torch.bfloat16, torch.float16) or X.dim() != 2:
        raise TypeError("X must be a 2-D bfloat16 or float16 tensor")
    _on_device(X, X=X)
    M, K = X.shape
    if W.dim() != 2:
        raise ValueError("W must be (N, K/2) bytes")
    N = W.shape[0]
    if K % 2 or kblock <= 0:
        raise ValueError("K must be even and kblock positive")
    _matrix("W", W, N, K // 2, (torch.uint8, getattr(torch, "float4_e2m1fn_x2", torch.uint8)))
    groups = -(-K // kblock)
    _matrix("SFW", SFW, N, groups, _E8M0)
    D, out = _product_out(X, M, N, C, D, out_dtype)
    _on_device(X, W=W, SFW=SFW, C=C, D=D)
    cp, ldc = _ptr_ld(C, N)
    _run("gemv_mxfp4", X.device, M, N, K, int(kblock), X.data_ptr(), _ld(X, K), _TYPES[X.dtype], W.data_ptr(),
         2 * _ld(W, K // 2), SFW.data_ptr(), _ld(SFW, groups), cp, ldc, D.data_ptr(), _ld(D, N), out)
    return D
