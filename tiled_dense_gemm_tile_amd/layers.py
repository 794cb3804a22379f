"""Binding of ``include/tilegemm_layers.h``: operators of a feed-forward
layer's linear parts.

Training: ``gemm_glu`` (with ``keep=True``) and ``gemm_glu_backward``, then
``clip_grads`` before the optimiser.  Serving: ``gemm_glu`` from one token on,
or ``int8_quantize`` and ``gemm_int8``.

Tensors are 2-D with a last stride of 1; the first stride is the leading
dimension.  Outputs not given are allocated.  Calls are enqueued on torch's
current stream of the tensors' GPU.
"""
from __future__ import annotations

import ctypes
from array import array

import torch

from . import _load
from .ops import _F32, _NONE, _TYPES, _device, _fast, _matrix, _new, _rows, _run, _vector, _workspace

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
_INT8 = (torch.int8,)


_entries = {}


def _entry(name):
    """The C function, called without ctypes' conversions where csrc/tensors.cpp
    is built."""
    f = _entries.get(name)
    if f is None:
        f = getattr(_load(), name)
        if _fast is not None:
            _fast.bind(name, ctypes.cast(f, ctypes.c_void_p).value)
            f = getattr(_fast, name)
        _entries[name] = f
    return f


def _act(name):
    if name not in ACTIVATIONS:
        raise ValueError("act must be one of %s" % ", ".join(ACTIVATIONS))
    return ACTIVATIONS[name]


def _type16(name, t):
    if t.dim() != 2 or (t.dtype != torch.bfloat16 and t.dtype != torch.float16):
        raise TypeError("%s must be a 2-D bfloat16 or float16 tensor" % name)
    return (t.dtype,)


def _copy_room(need, sizes, unit, workspace, dev, *operands):
    """(tensor to keep, pointer, bytes) of a product's workspace: given, or
    allocated here where rows that do not start on 16 bytes would be copied."""
    if workspace is None:
        at, off = 0, sizes[2]
        for p, ld in operands:
            at |= p
            off |= ld
        if at % 16 == 0 and off % unit == 0:
            return None, None, 0
        return _workspace(None, need(*sizes), dev)
    return _workspace(workspace, 0, dev)


def gemm_glu_workspace_bytes(M: int, F: int, K: int) -> int:
    """Workspace bytes with which :func:`gemm_glu` may copy operands whose rows
    do not start on 16 bytes (0: it would not)."""
    return _entry("gemm_glu_workspace_bytes")(M, F, K)


def gemm_glu(X, Wg, Wu, act="silu", H=None, G=None, U=None, keep=False, workspace=None):
    """Gated block of a feed-forward layer: H (M, F) = act(X @ Wg^T) * (X @
    Wu^T), X (M, K), Wg and Wu (F, K; two tensors, or the halves of one), all
    bfloat16 or all float16.  ``act``: "silu", "gelu", "gelu_tanh" or "relu".
    Sums and activation in fp32, H rounded once.  ``keep``, or G or U given:
    the two products are given out too, rounded, for
    :func:`gemm_glu_backward`.  ``workspace``: a device byte tensor, 256-byte
    aligned, of :func:`gemm_glu_workspace_bytes` bytes (allocated per call when
    not given and of use; a smaller one runs without copying operands whose
    rows do not start on 16 bytes).  Returns H, or (H, G, U) with those kept
    (None where one of G and U alone was given)."""
    own = _type16("X", X)
    dev = _device(X)
    M, K = X.shape
    if Wg.dim() != 2:
        raise ValueError("Wg must be 2-D")
    F = Wg.shape[0]
    x = _matrix("X", X, (M, K), own, dev)
    wg, wu = _matrix("Wg", Wg, (F, K), own, dev), _matrix("Wu", Wu, (F, K), own, dev)
    if H is None:
        H = _new((M, F), X.dtype, dev)
    if keep:
        G = _new((M, F), X.dtype, dev) if G is None else G
        U = _new((M, F), X.dtype, dev) if U is None else U
    g = _NONE if G is None else _matrix("G", G, (M, F), own, dev)
    u = _NONE if U is None else _matrix("U", U, (M, F), own, dev)
    workspace, *ws = _copy_room(gemm_glu_workspace_bytes, (M, F, K), 8, workspace, dev, x, wg, wu)
    _run(_entry("gemm_glu"), dev, M, F, K, *x, *wg, *wu, _TYPES[X.dtype], _act(act), *_matrix("H", H, (M, F), own, dev),
         *g, *u, *ws)
    return H if G is None and U is None else (H, G, U)


def gemm_glu_backward_workspace_bytes(M: int, F: int, K: int) -> int:
    """Workspace bytes :func:`gemm_glu_backward` needs."""
    return _entry("gemm_glu_backward_workspace_bytes")(M, F, K)


def gemm_glu_backward(dH, G, U, X, Wg, Wu, act="silu", Cg=None, Cu=None, dX=None, dWg=None, dWu=None,
                      grad_dtype=None, workspace=None, input_grad=True, weight_grad=True):
    """Gradients of :func:`gemm_glu` from the gradient dH (M, F) of H, with
    the G and U that it kept: dX (M, K) of X's type, dWg and dWu (F, K) of
    ``grad_dtype`` (X's type, the default, or float32), Cg and Cu of that type
    added to them (both or neither; Cg may be dWg and Cu dWu: gradients
    accumulated in place).  The gradients of G and U, the products' operands, are
    rounded to X's type: scale the loss so that float16 holds them.
    ``input_grad=False`` / ``weight_grad=False``: not
    computed, returned as None.  ``workspace``: a device byte tensor of at
    least :func:`gemm_glu_backward_workspace_bytes` bytes, 256-byte aligned
    (allocated per call when not given).  Returns (dX, dWg, dWu)."""
    own = _type16("X", X)
    dev = _device(X)
    M, K = X.shape
    if Wg.dim() != 2:
        raise ValueError("Wg must be 2-D")
    F = Wg.shape[0]
    if grad_dtype is None:
        grad_dtype = X.dtype if dWg is None else dWg.dtype
    if grad_dtype != torch.float32 and grad_dtype != X.dtype:
        raise TypeError("grad_dtype must be float32 or X's type")
    grad = (grad_dtype,)
    dh, g, u = _matrix("dH", dH, (M, F), own, dev), _matrix("G", G, (M, F), own, dev), _matrix("U", U, (M, F), own, dev)
    x = _matrix("X", X, (M, K), own, dev)
    wg, wu = _matrix("Wg", Wg, (F, K), own, dev), _matrix("Wu", Wu, (F, K), own, dev)
    dx = cg = cu = dwg = dwu = _NONE
    if input_grad:
        if dX is None:
            dX = _new((M, K), X.dtype, dev)
        dx = _matrix("dX", dX, (M, K), own, dev)
    elif dX is not None:
        raise ValueError("dX given with input_grad=False")
    if (Cg is None) != (Cu is None):
        raise ValueError("Cg and Cu are given both or neither")
    if weight_grad:
        if dWg is None:
            dWg = _new((F, K), grad_dtype, dev)
        if dWu is None:
            dWu = _new((F, K), grad_dtype, dev)
        dwg, dwu = _matrix("dWg", dWg, (F, K), grad, dev), _matrix("dWu", dWu, (F, K), grad, dev)
        if Cg is not None:
            cg, cu = _matrix("Cg", Cg, (F, K), grad, dev), _matrix("Cu", Cu, (F, K), grad, dev)
    elif not (dWg is dWu is Cg is Cu is None):
        raise ValueError("dWg, dWu, Cg or Cu given with weight_grad=False")
    workspace, *ws = _workspace(workspace, workspace is None and gemm_glu_backward_workspace_bytes(M, F, K), dev)
    _run(_entry("gemm_glu_backward"), dev, M, F, K, *dh, *g, *u, *x, *wg, *wu, _TYPES[X.dtype], _act(act), *dx, *cg, *cu,
         *dwg, *dwu, _TYPES[grad_dtype], *ws)
    return dX, dWg, dWu


def int8_quantize(X, Q=None, S=None):
    """X (rows, N) as 8-bit integers with one scale a row: S (rows,) float32 =
    max(max|x| / 127, 2^-126), Q (rows, N) int8 = x / S rounded to nearest
    even.  A row with a NaN or an infinity has codes 0 and the scale NaN.
    Returns (Q, S)."""
    shape, code, dev = _rows("X", X)
    x = _matrix("X", X, shape, (X.dtype,), dev)
    if Q is None:
        Q = _new(shape, torch.int8, dev)
    if S is None:
        S = _new(shape[0], torch.float32, dev)
    _run(_entry("int8_quantize"), dev, *shape, *x, code, *_matrix("Q", Q, shape, _INT8, dev),
         _vector("S", S, shape[0], _F32, dev))
    return Q, S


def gemm_int8_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace bytes with which :func:`gemm_int8` may copy operands whose rows
    do not start on 16 bytes (0: it would not)."""
    return _entry("gemm_int8_workspace_bytes")(M, N, K)


def gemm_int8(A, SA, B, SB, C=None, out_dtype=None, D=None, workspace=None):
    """D (M, N) = SA[m] * SB[n] * (A @ B^T) + C, A (M, K) and B (N, K) int8, SA
    (M,) and SB (N,) float32: the operands that :func:`int8_quantize` makes, of
    tokens and of a weight's channels.  The integer sums are exact (K below
    2^17).  ``out_dtype`` float32 (default), bfloat16 or float16; C of that
    type, (M, N) or (N,) (a bias); C may be D.  ``workspace`` as in
    :func:`gemm_glu`, of :func:`gemm_int8_workspace_bytes` bytes."""
    if A.dim() != 2 or A.dtype != torch.int8 or B.dim() != 2:
        raise TypeError("A and B must be 2-D int8 tensors")
    dev = _device(A)
    M, K = A.shape
    N = B.shape[0]
    a, b = _matrix("A", A, (M, K), _INT8, dev), _matrix("B", B, (N, K), _INT8, dev)
    sa, sb = _vector("SA", SA, M, _F32, dev), _vector("SB", SB, N, _F32, dev)
    if out_dtype is None:
        out_dtype = torch.float32 if D is None else D.dtype
    if out_dtype not in _TYPES:
        raise TypeError("out_dtype must be float32, bfloat16 or float16")
    own = (out_dtype,)
    if D is None:
        D = _new((M, N), out_dtype, dev)
    c = _NONE
    if C is not None:
        c = (_vector("C", C, N, own, dev), 0) if C.dim() == 1 else _matrix("C", C, (M, N), own, dev)
    workspace, *ws = _copy_room(gemm_int8_workspace_bytes, (M, N, K), 16, workspace, dev, a, b)
    _run(_entry("gemm_int8"), dev, M, N, K, *a, sa, *b, sb, *c, *_matrix("D", D, (M, N), own, dev), _TYPES[out_dtype],
         *ws)
    return D


# ---- gradients ------------------------------------------------------------------

def _dense(t):
    """Whether the tensor's elements fill one piece of memory, in any order."""
    if t.is_contiguous():
        return True
    want = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n > 1):
        if stride != want:
            return False
        want *= size
    return True


def _gradients(name, grads):
    """(device, whether all are contiguous, addresses, sizes, types) of a list
    of tensors: the arrays that the C calls read."""
    if _fast is not None and (found := _fast.gradients(grads)) is not None:
        dev, at, sizes, types = found
        return dev, True, at, memoryview(sizes).cast("q"), types
    if not grads:
        raise ValueError("no %s" % name)
    dev = _device(grads[0])
    if {t.get_device() for t in grads} != {dev}:       # (-1 of a host tensor)
        raise ValueError("%s must be device tensors on cuda:%d" % (name, dev))
    whole = all([t.is_contiguous() for t in grads])
    if not whole and not all([_dense(t) for t in grads]):
        raise ValueError("%s must each fill one piece of memory" % name)
    try:
        types = array("i", [_TYPES[t.dtype] for t in grads])
    except KeyError:
        raise TypeError("%s must be float32, bfloat16 or float16 tensors" % name) from None
    return dev, whole, array("q", [t.data_ptr() for t in grads]), array("q", [t.numel() for t in grads]), types


def _twice(at, sizes):
    """Whether two tensors with elements start at the same address."""
    if isinstance(at, bytes):
        at = memoryview(at).cast("q")
    if len(set(at)) == len(at):
        return False
    at = [a for a, n in zip(at, sizes) if n]
    return len(set(at)) != len(at)


def _at(a):
    """What a call takes as the address of the array (a bytes object as it is)."""
    if isinstance(a, memoryview):
        return a.obj
    return a if isinstance(a, bytes) else a.buffer_info()[0]


def grad_workspace_bytes(n: int) -> int:
    """Workspace bytes :func:`grad_norm` and :func:`clip_grads` need for n
    tensors."""
    return _entry("grad_workspace_bytes")(n)


def grad_norm(grads, norm=None, workspace=None):
    """Norm of all gradients taken together (float32, no dimension), summed
    in fp64: the root of the sum of their elements' squares.  ``grads``:
    tensors of float32, bfloat16 or float16, of any shapes, each filling one
    piece of memory.  ``workspace``: a device byte tensor of at least
    :func:`grad_workspace_bytes` bytes, 256-byte aligned (allocated per call
    when not given)."""
    grads = list(grads)
    dev, _, at, sizes, types = _gradients("gradients", grads)
    norm, to = _norm_out(norm, dev)
    workspace, *ws = _workspace(workspace, workspace is None and grad_workspace_bytes(len(grads)), dev)
    _run(_entry("grad_norm"), dev, len(grads), _at(at), _at(sizes), _at(types), to, *ws)
    return norm


def _norm_out(norm, dev):
    if norm is None:
        norm = _new((), torch.float32, dev)
    return norm, _scalar("norm", norm, dev)


def _scalar(name, t, dev):
    if t.dtype != torch.float32 or t.numel() != 1 or t.get_device() != dev:
        raise ValueError("%s must be one float32 on cuda:%d" % (name, dev))
    return t.data_ptr()


def clip_grads(grads, max_norm, out=None, norm=None, given=None, workspace=None):
    """Every gradient times min(1, max_norm / (norm + 1e-6)), in place or into
    ``out`` (tensors of the same sizes and types, contiguous where the
    gradients are, else of the same strides).  The norm is that
    of :func:`grad_norm`, computed here, or ``given``: one float32 on the GPU,
    such as a norm whose square the ranks have summed.  Returns the norm
    (``given`` where it was).  An infinite ``max_norm`` leaves every gradient as
    it is (unless the norm is NaN).  No two gradients may share memory."""
    grads = list(grads)
    dev, whole, at, sizes, types = _gradients("gradients", grads)
    if _twice(at, sizes):
        raise ValueError("the same gradient is given twice")
    to = at
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError("out must hold one tensor for each gradient")
        odev, owhole, to, osizes, otypes = _gradients("out", out)
        if odev != dev:
            raise ValueError("out must be device tensors on cuda:%d" % dev)
        if otypes != types or osizes != sizes or (not (whole and owhole) and any(
                [o.shape != t.shape or (o.stride() != t.stride() and t.numel() > 1) for t, o in zip(grads, out)])):
            raise ValueError("out must have the gradients' sizes and types, and strides where those are not contiguous")
        if _twice(to, sizes):
            raise ValueError("the same result is given twice")
    if given is None:
        norm, into = _norm_out(norm, dev)
        read = None
        workspace, *ws = _workspace(workspace, workspace is None and grad_workspace_bytes(len(grads)), dev)
    else:
        if norm is not None:
            raise ValueError("norm is an output: give either it or given")
        norm, read, into, ws = given, _scalar("given", given, dev), None, (None, 0)
    _run(_entry("grad_clip"), dev, len(grads), _at(at), _at(to), _at(sizes), _at(types), max_norm, read, into, *ws)
    return norm
