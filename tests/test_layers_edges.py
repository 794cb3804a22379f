"""Edges of the feed-forward layer's operators on the CPU: memory that a call
may not share, sizes next to the limits (no compute call is made)."""
from test_layers_abi import MB, P, Q, UNSUPPORTED, bwd, grads

import tiled_dense_gemm_tile_amd as tg


def test_norm_and_workspace_apart_from_the_gradients():
    """What grad_norm writes lies neither in a gradient nor in its workspace."""
    room = tg.grad_workspace_bytes(2)
    for over in (dict(norm=P), dict(norm=P + 16), dict(norm=P + MB + 76), dict(ws=P), dict(ws=P + MB), dict(at=(P, Q + MB + 64)),
                 dict(at=(Q + MB + room - 4, P)), dict(norm=Q + MB), dict(norm=Q + MB + room - 4)):
        assert grads(clip=False, **over) == UNSUPPORTED, over


def test_clip_writes_apart_from_what_it_reads():
    """With results of their own: the norm and the workspace lie in no gradient either, and, in place too, not in each
    other."""
    room, apart = tg.grad_workspace_bytes(2), dict(out=(Q + 2 * MB, Q + 3 * MB))
    for over in (dict(norm=P), dict(norm=P + 16), dict(norm=P + MB + 76), dict(ws=P), dict(ws=P + MB), dict(at=(P, Q + MB + 64)),
                 dict(at=(Q + MB + room - 4, P)), dict(given=Q + 4 * MB, norm=P + 16), dict(given=Q + 4 * MB, norm=P + MB + 76)):
        assert grads(**over, **apart) == UNSUPPORTED, over
    for over in (dict(norm=Q + MB), dict(norm=Q + MB + room - 4)):
        assert grads(**over) == UNSUPPORTED, over
        assert grads(**over, **apart) == UNSUPPORTED, over


def test_glu_backward_pieces():
    """More than 2^24 pieces of 64 x 64 are refused: M x F, M x K and twice F x K."""
    room = dict(ws=1 << 50, wb=1 << 60, lddh=1 << 19, ldg=1 << 19, ldu=1 << 19, G=1 << 42, U=1 << 43, X=1 << 44, Wg=1 << 45, Wu=1 << 46,
                dX=1 << 47, dWg=1 << 48, dWu=1 << 49)
    for m, f, k, ld in ((1 << 20, 1 << 16, 64, 64), (1 << 20, 64, 1 << 16, 1 << 16), (64, 1 << 18, 1 << 17, 1 << 17)):
        sizes = dict(M=m, F=f, K=k, ldx=ld, ldwg=ld, ldwu=ld, lddx=ld, lddwg=ld, lddwu=ld)
        assert bwd(**sizes, **room) == UNSUPPORTED
