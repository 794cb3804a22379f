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

from . import OUT_BF16, OUT_F32, _check, _load

try:                                                   # the checks below in C++ (csrc/tensors.cpp): quicker, not needed
    from . import _tensors as _fast
except ImportError:
    _fast = None

_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_E4M3 = (torch.float8_e4m3fn, torch.uint8)
_E8M0 = (torch.float8_e8m0fnu, torch.uint8)
_E2M1 = (torch.uint8, torch.float4_e2m1fn_x2)
_F32 = (torch.float32,)
_NONE = (None, 0)
_LD_LIMIT = 1 << 21                                    # elements of 4 bytes: the products' rows are below 8 MiB
_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _run(f, dev, *args):
    """The C call on torch's current stream of GPU ``dev``, with ``dev``
    current (a NULL stream means the current device's)."""
    stream = _current_stream(dev)
    if _current_device() == dev:
        status = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = f(*args, stream)
    if status:
        _check(status)


def _device(X):
    """Index of the tensor's GPU."""
    if not X.is_cuda:
        raise ValueError("the tensors must be device tensors")
    return X.get_device()


_GPUS = [torch.device("cuda", i) for i in range(64)]


def _new(shape, dtype, dev):
    t = None if _fast is None else _fast.empty(shape, dtype, dev)
    return torch.empty(shape, dtype=dtype, device=_GPUS[dev]) if t is None else t


def _matrix(name, t, shape, dtypes, dev):
    """(pointer, leading dimension) of a matrix, checked."""
    if _fast is not None and (found := _fast.matrix(t, shape, dtypes, dev)) is not None:
        return found
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s" % (name, " or ".join(str(d) for d in dtypes)))
    if t.shape != shape:
        raise ValueError("%s must be (%d, %d)" % (name, shape[0], shape[1]))
    if t.get_device() != dev:                          # (-1 of a host tensor)
        raise ValueError("%s must be a device tensor on cuda:%d" % (name, dev))
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError("%s: the last stride must be 1" % name)
    if shape[0] <= 1 and not shape[1] <= ld < _LD_LIMIT:  # (of one row any will do: x[:, -1] of a long batch of one)
        ld = shape[1]
    return t.data_ptr(), ld


def _vector(name, t, n, dtypes, dev):
    """Pointer of a contiguous vector, checked."""
    if _fast is not None and (found := _fast.vector(t, n, dtypes, dev)) is not None:
        return found
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s" % (name, " or ".join(str(d) for d in dtypes)))
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be a contiguous vector of %d" % (name, n))
    if t.get_device() != dev:                          # (-1 of a host tensor)
        raise ValueError("%s must be a device tensor on cuda:%d" % (name, dev))
    return t.data_ptr()


def _rows(name, X):
    """(shape, type code, device) of the first matrix of a row operator."""
    if X.dim() != 2 or X.dtype not in _TYPES:
        raise TypeError("%s must be a 2-D float32, bfloat16 or float16 tensor" % name)
    return tuple(X.shape), _TYPES[X.dtype], _device(X)


def _scaled_out(shape, dev, Q, SF):
    rows, N = shape
    if N % 32:
        raise ValueError("block-scaled rows hold a multiple of 32 elements")
    if Q is None:
        Q = _new(shape, torch.float8_e4m3fn, dev)
    if SF is None:
        SF = _new((rows, N // 32), torch.float8_e8m0fnu, dev)
    return Q, SF, _matrix("Q", Q, shape, _E4M3, dev) + _matrix("SF", SF, (rows, N // 32), _E8M0, dev)


def _workspace(t, need, dev):
    """(tensor to keep, pointer, bytes) of a workspace given or allocated here."""
    if t is None:
        if not need:
            return None, None, 0
        t = _new(need, torch.uint8, dev)
    elif t.get_device() != dev or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor on cuda:%d" % dev)
    return t, t.data_ptr(), t.numel() * t.element_size()


def mxfp8_quantize(X, Q=None, SF=None):
    """X (rows, N) as block-scaled rows: e4m3 codes Q (rows, N) and e8m0
    scales SF (rows, N/32), as :func:`gemm_mxfp8` takes an operand.  N must
    be a multiple of 32.  The scale of a block is the least power of two that
    clips none of its elements.  Returns (Q, SF)."""
    shape, code, dev = _rows("X", X)
    x = _matrix("X", X, shape, (X.dtype,), dev)
    Q, SF, out = _scaled_out(shape, dev, Q, SF)
    _run(_load().mxfp8_quantize, dev, *shape, *x, code, *out)
    return Q, SF


def _norm(f, X, W, eps, residual, H, rstd, shape, code, dev, out):
    """The norm's call; returns (H, rstd)."""
    own = (X.dtype,)
    x = _matrix("X", X, shape, own, dev)
    w = _vector("W", W, shape[1], (X.dtype, torch.float32), dev)
    r = _NONE
    if residual is not None:
        r = _matrix("residual", residual, shape, own, dev)
        if H is None:
            H = _new(shape, X.dtype, dev)
    h = _NONE if H is None else _matrix("H", H, shape, own, dev)
    if rstd is None:
        rstd = _new(shape[0], torch.float32, dev)
    _run(f, dev, *shape, *x, *r, code, w, _TYPES[W.dtype], eps, *h, *out, _vector("rstd", rstd, shape[0], _F32, dev))
    return X if H is None else H, rstd


def rmsnorm(X, W, eps, residual=None, Y=None, H=None, rstd=None):
    """Root-mean-square norm of each row of H = X + residual (rounded to X's
    type; X itself without a residual): Y = H * W * rstd, rstd = 1 /
    sqrt(mean(H^2) + eps).  W (N,) of X's type or float32.  H may be given as
    X or the residual (in place), and so may Y unless H is the same.
    Returns (Y, H, rstd), H being X when there is no residual and no H (None
    where Y has overwritten it)."""
    shape, code, dev = _rows("X", X)
    if Y is None:
        Y = _new(shape, X.dtype, dev)
    out = _matrix("Y", Y, shape, (X.dtype,), dev)
    H, rstd = _norm(_load().rmsnorm, X, W, eps, residual, H, rstd, shape, code, dev, out)
    return Y, None if H is X and out[0] == X.data_ptr() and X.numel() else H, rstd


def rmsnorm_mxfp8(X, W, eps, residual=None, Q=None, SF=None, H=None, rstd=None):
    """:func:`rmsnorm` with the result as block-scaled rows (see
    :func:`mxfp8_quantize`): the operand of :func:`gemm_mxfp8` and the 8-bit
    copy that :func:`gemm_wgrad_mxfp8` reads in the backward pass.  Returns
    (Q, SF, H, rstd)."""
    shape, code, dev = _rows("X", X)
    Q, SF, out = _scaled_out(shape, dev, Q, SF)
    return (Q, SF, *_norm(_load().rmsnorm_mxfp8, X, W, eps, residual, H, rstd, shape, code, dev, out))


def rmsnorm_backward_workspace_bytes(rows: int, N: int) -> int:
    """Workspace bytes :func:`rmsnorm_backward` needs for dW."""
    return _load().rmsnorm_backward_workspace_bytes(rows, N)


def rmsnorm_backward(dY, H, W, rstd, dH=None, dX=None, dW=None, workspace=None, weight_grad=True):
    """Gradients of :func:`rmsnorm` / :func:`rmsnorm_mxfp8` from the gradient
    dY of its result: dX (dY's type; the gradient of X and of the residual
    alike) and dW (float32; None with ``weight_grad=False``).  H and rstd as
    the forward call returned them; ``dH``: the gradient that reaches H from
    elsewhere, added to dX.  dX may be given as dY or dH (in place).
    ``workspace``: a device byte tensor of at least
    :func:`rmsnorm_backward_workspace_bytes` bytes, 256-byte aligned
    (allocated per call when not given).  Returns (dX, dW)."""
    shape, code, dev = _rows("dY", dY)
    rows, N = shape
    own = (dY.dtype,)
    dy = _matrix("dY", dY, shape, own, dev)
    h = _matrix("H", H, shape, own, dev)
    w = _vector("W", W, N, (dY.dtype, torch.float32), dev)
    s = _vector("rstd", rstd, rows, _F32, dev)
    dh = _NONE if dH is None else _matrix("dH", dH, shape, own, dev)
    if dX is None:
        dX = _new(shape, dY.dtype, dev)
    dx = _matrix("dX", dX, shape, own, dev)
    dw, ws = None, (None, 0)
    if weight_grad:
        if dW is None:
            dW = _new(N, torch.float32, dev)
        dw = _vector("dW", dW, N, _F32, dev)
        workspace, *ws = _workspace(workspace, workspace is None and rmsnorm_backward_workspace_bytes(rows, N), dev)
    elif dW is not None:
        raise ValueError("dW given with weight_grad=False")
    _run(_load().rmsnorm_backward, dev, rows, N, *dy, *h, code, w, _TYPES[W.dtype], s, *dh, *dx, dw, *ws)
    return dX, dW


def _product_out(shape, dev, C, D, out_dtype):
    """(D, output type code, C's pointer and leading dimension, D's)."""
    if out_dtype is None:
        out_dtype = torch.float32
    elif out_dtype != torch.float32 and out_dtype != torch.bfloat16:
        raise TypeError("out_dtype must be float32 or bfloat16")
    if D is None:
        D = _new(shape, out_dtype, dev)
    c = _NONE if C is None else _matrix("C", C, shape, (out_dtype,), dev)
    return D, OUT_BF16 if out_dtype == torch.bfloat16 else OUT_F32, c + _matrix("D", D, shape, (out_dtype,), dev)


def gemm_wgrad_mxfp8_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace bytes with which :func:`gemm_wgrad_mxfp8` may cut K or copy A
    (0: it would not)."""
    return _load().gemm_wgrad_mxfp8_workspace_bytes(M, N, K)


def gemm_wgrad_mxfp8(dY, Q, SF, C=None, out_dtype=None, D=None, workspace=None):
    """Weight gradient from an 8-bit activation: D (M, N) = dY^T @ X + C, dY
    (K tokens, M) bfloat16 and X (K, N) given as block-scaled rows Q, SF
    (:func:`mxfp8_quantize`, :func:`rmsnorm_mxfp8`).  ``out_dtype`` float32
    (default) or bfloat16, C of that type; C may be D (gradient
    accumulation).  ``workspace``: a device byte tensor, 256-byte aligned, of
    :func:`gemm_wgrad_mxfp8_workspace_bytes` bytes (allocated per call when
    not given; a smaller one runs without cutting K or moving dY's rows to 16
    bytes)."""
    if dY.dtype != torch.bfloat16 or dY.dim() != 2:
        raise TypeError("dY must be a 2-D bfloat16 tensor")
    if Q.dim() != 2 or Q.shape[1] % 32:
        raise ValueError("Q must be (K, N) with N a multiple of 32")
    dev = _device(dY)
    K, M = dY.shape
    N = Q.shape[1]
    a = _matrix("dY", dY, (K, M), (torch.bfloat16,), dev)
    b = _matrix("Q", Q, (K, N), _E4M3, dev)
    s = _matrix("SF", SF, (K, N // 32), _E8M0, dev)
    D, out, cd = _product_out((M, N), dev, C, D, out_dtype)
    workspace, *ws = _workspace(workspace, workspace is None and gemm_wgrad_mxfp8_workspace_bytes(M, N, K), dev)
    _run(_load().gemm_wgrad_mxfp8, dev, M, N, K, *a, *b, *s, *cd, out, *ws)
    return D


def gemv_mxfp4_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace bytes with which :func:`gemv_mxfp4` may cut K (0: it would
    not)."""
    return _load().gemv_mxfp4_workspace_bytes(M, N, K)


def gemv_mxfp4(X, W, SFW, kblock=32, C=None, out_dtype=None, D=None, workspace=None):
    """A few rows times 4-bit weights: D (M, N) = X @ W^T + C, X (M, K)
    bfloat16 or float16, W (N, K/2) bytes of two e2m1 codes and SFW (N,
    ceil(K / kblock)) e8m0 codes, as :func:`gemm_mxfp4` and
    :func:`gemm_mx_kblock` take B and SFB.  X is not quantised.  Made for up
    to 16 rows, right for any number.  ``out_dtype`` float32 (default) or
    bfloat16; C of that type may be D.  ``workspace``: a device byte tensor,
    256-byte aligned, of :func:`gemv_mxfp4_workspace_bytes` bytes (allocated
    per call when not given; a smaller one runs without cutting K)."""
    if X.dim() != 2 or (X.dtype != torch.bfloat16 and X.dtype != torch.float16):
        raise TypeError("X must be a 2-D bfloat16 or float16 tensor")
    dev = _device(X)
    M, K = X.shape
    if W.dim() != 2 or K % 2 or kblock <= 0:
        raise ValueError("W must be (N, K/2) bytes, K even and kblock positive")
    N = W.shape[0]
    x = _matrix("X", X, (M, K), (X.dtype,), dev)
    wp, ldw = _matrix("W", W, (N, K // 2), _E2M1, dev)
    s = _matrix("SFW", SFW, (N, -(-K // kblock)), _E8M0, dev)
    D, out, cd = _product_out((M, N), dev, C, D, out_dtype)
    L = _load()
    workspace, *ws = _workspace(workspace, workspace is None and L.gemv_mxfp4_workspace_bytes(M, N, K), dev)
    _run(L.gemv_mxfp4, dev, M, N, K, kblock, *x, _TYPES[X.dtype], wp, 2 * ldw, *s, *cd, out, *ws)
    return D
