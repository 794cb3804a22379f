"""The waits of the four-wave weight-gradient kernel, checked in the gfx950
assembly of its source (CPU only: compiled, never run).

A K tile ends with s_waitcnt vmcnt(n) and a barrier, after which A's next
tile is read from LDS.  n counts on what the tiles issue after that tile's
loads: were a load left out of one copy of the unrolled loop, n would be too
many and the tile could be read before it has landed.  Here every path through
the kernel is followed with the queue of outstanding vector-memory operations
(they return in order), of which a wait leaves the youngest n; only the waits
right before the barriers are counted, so that the others, which come and go
with the compiler's choices, carry nothing."""
import os
import re
import shutil
import subprocess

import pytest

from tiled_dense_gemm_tile_amd import build as B

pytestmark = pytest.mark.skipif(shutil.which(B.HIPCC) is None and not os.path.exists(B.HIPCC),
                                reason="hipcc not available")

KERNEL = "gemm_wgrad_w4_kernelILb%dELi%dE"
# per tile size: A's loads a K tile and wave, K tiles from their issue to their use
A_LOADS, AHEAD = {8: 8, 4: 4}, {8: 1, 4: 2}


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("asm") / "wgrad.s")
    subprocess.run([B.HIPCC] + B.FLAGS + ["-S", "--cuda-device-only", os.path.join(B.CSRC, "wgrad.hip"), "-o", out],
                   check=True, capture_output=True)
    return open(out).read()


def blocks_of(text, name):
    """Basic blocks of a kernel: {label: (instructions, labels that follow)}, the first one's label."""
    body = re.search(r"^(\w*%s\w*):.*?^\.Lfunc_end" % re.escape(name), text, re.M | re.S).group(0)
    blocks, label, first, fresh = {}, "entry", "entry", 0
    ins, ended = [], False

    def close(nxt, falls):
        blocks[label][1].extend([nxt] if falls else [])

    blocks[label] = (ins, [])
    for line in body.splitlines()[1:]:
        line = line.split(";")[0].strip()
        m = re.match(r"(\.LBB\w+):$", line)
        if m:
            close(m.group(1), not ended)
            label, ins, ended = m.group(1), [], False
            blocks[label] = (ins, [])
        elif line and not line.startswith("."):
            op = line.split()[0]
            ins.append(line)
            if op.startswith("s_cbranch"):
                blocks[label][1].append(line.split()[-1])
                fresh += 1
                close("after%d" % fresh, True)
                label, ins, ended = "after%d" % fresh, [], False
                blocks[label] = (ins, [])
            elif op == "s_branch":
                blocks[label][1].append(line.split()[-1])
                ended = True
            elif op == "s_endpgm":
                ended = True
    return blocks, first


VMEM = re.compile(r"(buffer|global|flat|scratch)_(load|store|atomic)")


def count_of(line):
    """The vector-memory count of a wait (63: none)."""
    m = re.search(r"vmcnt\((\d+)\)", line)
    return int(m.group(1)) if m else 63


def walk(text, name, loads, ahead, visit):
    """Follows every path; `visit(nth, queue, wait, least)` at each barrier, with the queue after its wait, that wait's
    count and the least count of the waits since the barrier before.  An entry of the queue is the number of barriers until
    it has to have landed (0: any time); nth counts the barriers up to two."""
    blocks, first = blocks_of(text, name)
    # (block, queue, barriers passed up to two, direct loads since the last one, least count since it)
    todo, seen, barriers = [(first, (), 0, 0, 63)], set(), 0
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        assert len(seen) < 200000
        label, queue, passed, direct, least = state
        ins, after = blocks[label]
        for i, line in enumerate(ins):
            if VMEM.match(line):
                due = 0
                if line.endswith(" lds"):
                    if passed:
                        due = ahead if direct < loads else 0
                    else:                              # the first tiles, before the first barrier
                        due = direct // loads + 1 if direct < loads * ahead else 0
                    direct += 1
                queue += (due,)
                queue = queue[-64:]
            elif line.startswith("s_waitcnt") and "vmcnt" in line and not ins[i + 1:i + 2] == ["s_barrier"]:
                least = min(least, count_of(line))
            elif line.startswith("s_barrier"):
                n = count_of(ins[i - 1]) if i else 63
                if n < len(queue):
                    queue = queue[len(queue) - n:]
                visit(passed, queue, n, least)
                barriers += 1
                queue = tuple(max(d - 1, 0) for d in queue)
                passed, direct, least = min(passed + 1, 2), 0, 63
        todo.extend((b, queue, passed, direct, least) for b in after)
    return barriers


@pytest.mark.parametrize("tile", [8, 4])
@pytest.mark.parametrize("bf16", [0, 1])
def test_a_tile_has_landed_before_it_is_read(assembly, tile, bf16):
    def visit(nth, queue, wait, least):
        assert 1 not in queue, "A's next tile may still be on its way behind this barrier"

    assert walk(assembly, KERNEL % (bf16, tile), A_LOADS[tile], AHEAD[tile], visit) > 3


@pytest.mark.parametrize("tile", [8, 4])
@pytest.mark.parametrize("bf16", [0, 1])
def test_no_wait_inside_a_tile_is_longer_than_its_last(assembly, tile, bf16):
    """The loads of tiles ahead stay in flight through a tile: the compiler's own waits, for B's codes and scales, ask
    for no more than the wait at its end."""
    found = []

    def visit(nth, queue, wait, least):
        # (the first tile waits for codes loaded right before it; no count, or none left: behind the last tile)
        if nth == 2 and 0 < wait < 63:
            found.append(wait)
            assert least >= wait

    walk(assembly, KERNEL % (bf16, tile), A_LOADS[tile], AHEAD[tile], visit)
    assert found


def test_k_tiles_up_to_the_largest_k(tmp_path):
    """The count of K tiles at the ends of K's range, by the compiler (an overflow is an error there)."""
    src = tmp_path / "count.hip"
    src.write_text('#include "gemm_wgrad_w4.hpp"\n' + "".join(
        "static_assert(tg::k_tiles(%d, 64) == %d);\n" % (k, -(-k // 64))
        for k in (1, 63, 64, 65, 8200, 2 ** 31 - 65, 2 ** 31 - 64, 2 ** 31 - 63, 2 ** 31 - 1)))
    subprocess.run([B.HIPCC] + B.FLAGS + ["-I" + B.CSRC, "--cuda-host-only", "-fsyntax-only", str(src)], check=True,
                   capture_output=True)
    text = open(os.path.join(B.CSRC, "gemm_wgrad_w4.hpp")).read()
    assert text.count("k_tiles(K, KT)") == 1 and "K + KT" not in text
