"""The waits of the 256 x 256-tile products, checked in the gfx950 assembly of
their sources (CPU only: compiled, never run).

Operands come by direct loads into LDS, which nothing but a count of outstanding
vector-memory operations says to have landed: a K tile's barrier leaves one
operation in flight where lines are brought ahead (that one; with three slots
also the next but one K tile's loads), the barrier before the next output tile
leaves the finished tile's stores.  Here every path through
the kernels is followed with the queue of outstanding operations (they return in
order): none of those loads may be in it at a barrier, and nothing that writes
LDS at the kernel's end, where the LDS is another workgroup's next."""
import os
import re
import shutil
import subprocess

import pytest

from test_wgrad_waits import VMEM, blocks_of, count_of
from tiled_dense_gemm_tile_amd import build as B

pytestmark = pytest.mark.skipif(shutil.which(B.HIPCC) is None and not os.path.exists(B.HIPCC),
                                reason="hipcc not available")

# (The kernel of two products has the same body; its paths by which product it is are too many here.)
# An epilogue of which it is known, when it is compiled, whether its results lie in whole pieces and whether they are added
# to something: the kernels choose at run time, and paths that mix the one's stores with the other's wait do not exist.
HEAD = """
#include "prod_w4.hpp"
namespace tg {
template <class E, bool V, bool A> struct Known : E {
    static constexpr bool vec = V, add = A;
};
#define ONE(T, PAIR, AHEAD, E)                                                                                        \\
    template __global__ void prod_w4_kernel<T, PAIR, AHEAD, Known<E, true, false>>(ProdArgs, Known<E, true, false>); \\
    template __global__ void prod_w4_kernel<T, PAIR, AHEAD, Known<E, false, false>>(ProdArgs, Known<E, false, false>);
#define ADDING(T, PAIR, AHEAD, E)                                                                                     \\
    template __global__ void prod_w4_kernel<T, PAIR, AHEAD, Known<E, true, true>>(ProdArgs, Known<E, true, true>);    \\
    template __global__ void prod_w4_kernel<T, PAIR, AHEAD, Known<E, false, true>>(ProdArgs, Known<E, false, true>);
#define NARROW(T, PAIR, E, ...)                                                                                          \\
    template __global__ void prod_w4_kernel<T, PAIR, true, Known<E, __VA_ARGS__>, 4>(ProdArgs, Known<E, __VA_ARGS__>);   \\
    template __global__ void prod_w4_kernel<T, PAIR, true, Known<E, __VA_ARGS__>, 4, 4>(ProdArgs, Known<E, __VA_ARGS__>);
"""
# compiled apart, at the same time
PARTS = [
    ["ONE(1, true, true, GluEpi<1>)", "ONE(2, false, true, PlainEpi<2>)", "NARROW(1, true, GluEpi<1>, true, false)", "NARROW(1, false, PlainEpi<0>, false, true)"],
    ["ONE(2, true, true, GluEpi<2>)", "ADDING(3, false, false, Int8Epi<0>)", "NARROW(2, true, GluEpi<2>, false, false)", "NARROW(2, false, PlainEpi<2>, true, true)"],
    ["ONE(3, false, false, Int8Epi<0>)", "ADDING(3, false, false, Int8Epi<1>)", "NARROW(3, false, Int8Epi<0>, true, true)", "NARROW(2, false, PlainEpi<2>, true, false)"],
    ["ONE(3, false, false, Int8Epi<1>)", "ADDING(1, false, true, PlainEpi<0>)", "NARROW(3, false, Int8Epi<1>, false, true)"],
    ["ONE(1, false, true, PlainEpi<0>)", "ADDING(2, false, true, PlainEpi<2>)", "NARROW(3, false, Int8Epi<1>, true, false)"],
]


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    d = tmp_path_factory.mktemp("asm")
    runs = []
    for i, part in enumerate(PARTS):
        (d / ("w4_%d.hip" % i)).write_text(HEAD + "\n".join(part) + "\n}\n")
        runs.append(subprocess.Popen([B.HIPCC] + B.FLAGS + ["-I" + B.CSRC, "-S", "--cuda-device-only", str(d / ("w4_%d.hip" % i)),
                                                            "-o", str(d / ("w4_%d.s" % i))], stderr=subprocess.DEVNULL))
    assert [r.wait() for r in runs] == [0] * len(runs)
    return "".join((d / ("w4_%d.s" % i)).read_text() for i in range(len(PARTS)))


def follow(text, name, at_barrier, at_end):
    """Every path, with the queue of outstanding operations: 2 a load of 16 bytes a lane into LDS (3 behind the next
    barrier, 4 behind the one after it, ...), 1 a smaller one, 0 any other.  Only the queue from its oldest LDS load on is kept."""
    blocks, first = blocks_of(text, name)
    todo, seen, barriers = [(first, ())], set(), 0
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        assert len(seen) < 400000
        label, queue = state
        ins, after = blocks[label]
        for line in ins:
            if VMEM.match(line):
                queue += ((2 if "dwordx4" in line else 1) if line.endswith(" lds") else 0,)
            elif line.startswith("s_waitcnt"):
                n = count_of(line)
                queue = queue[len(queue) - n:] if 0 < n < len(queue) else queue if n else ()
            elif line.startswith("s_barrier"):
                at_barrier(name, queue)
                queue = tuple(q + 1 if q >= 2 else q for q in queue)
                barriers += 1
            elif line.startswith("s_endpgm"):
                at_end(queue)
            while queue and queue[0] == 0:
                queue = queue[1:]
            if len(queue) > 96:                        # (an LDS load this old is outstanding for good)
                queue = queue[:1] + queue[-95:]
        todo.extend((b, queue) for b in after)
    return barriers


def at_barrier(name, queue):
    """256 x 256 tiles: the next K tile is the last one issued.  256 x 128 and 128 x 128: one and two more, of 12 and 8
    loads each, are on their way, the latest issued since the barrier before (at the start all of them)."""
    ahead, loads = {"ELi8ELi8EEEv": (0, 0), "ELi4ELi8EEEv": (1, 12), "ELi4ELi4EEEv": (2, 8)}[re.search(r"(ELi\dELi\dEEEv)", name).group(1)]
    late = "an operand's load may still be on its way behind this barrier"
    assert all(q < 2 + ahead for q in queue if q >= 2), late
    assert sum(q >= 2 for q in queue) <= ahead * loads, late


def at_end(queue):
    assert not any(queue), "a load may write LDS after the workgroup's end"


def kernels(text):
    return sorted(set(re.findall(r"^(_ZN2tg\w*prod_w4_\w+):", text, re.M)))


def test_operands_have_landed_at_every_barrier(assembly):
    names = kernels(assembly)
    assert len(names) == 36
    for name in names:
        assert follow(assembly, name, at_barrier, at_end) > 4, name


def test_the_check_sees_waits_that_are_too_short(assembly):
    """The same text with one operation more left in flight, at the K tiles' ends or behind the results."""
    for kernel, wait, longer in (("prod_w4_kernelILi3ELb0ELb0ENS_5KnownINS_7Int8EpiILi1EEELb1ELb0EEELi8", 0, 1),
                                 ("prod_w4_kernelILi1ELb1ELb1ENS_5KnownINS_6GluEpiILi1EEELb1ELb0EEELi8", 1, 2),
                                 ("prod_w4_kernelILi1ELb1ELb1ENS_5KnownINS_6GluEpiILi1EEELb1ELb0EEELi8", 16, 17),
                                 ("prod_w4_kernelILi2ELb0ELb1ENS_5KnownINS_8PlainEpiILi2EEELb1ELb0EEELi4ELi8", 14, 15),
                                 ("prod_w4_kernelILi2ELb0ELb1ENS_5KnownINS_8PlainEpiILi2EEELb1ELb0EEELi4ELi8", 13, 14),
                                 ("prod_w4_kernelILi2ELb0ELb1ENS_5KnownINS_8PlainEpiILi2EEELb1ELb0EEELi4ELi4", 19, 20),
                                 ("prod_w4_kernelILi2ELb0ELb1ENS_5KnownINS_8PlainEpiILi2EEELb1ELb0EEELi4ELi4", 18, 19)):
        name = [k for k in kernels(assembly) if kernel in k][0]
        with pytest.raises(AssertionError):
            follow(assembly.replace("vmcnt(%d)" % wait, "vmcnt(%d)" % longer), name, at_barrier, at_end)
