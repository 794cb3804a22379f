"""The waits of the kernel of two products in one launch, checked as those of
the others in the gfx950 assembly (CPU only: compiled, never run).

Which of the two products a workgroup computes is known at run time only; paths
that mix the one's results with the other's waits do not exist.  The source is
compiled once for each, with that one line of it a constant."""
import os
import re
import shutil
import subprocess

import pytest

from test_layers_waits import HEAD, at_end, follow
from tiled_dense_gemm_tile_amd import build as B

pytestmark = pytest.mark.skipif(shutil.which(B.HIPCC) is None and not os.path.exists(B.HIPCC),
                                reason="hipcc not available")

WHICH = "const bool second = (int)blockIdx.x >= q.split;"
# (first product's results in whole pieces; second's type, in whole pieces, added to something)
FORMS = [(1, "true", 0, "true", "true"), (1, "false", 0, "false", "true"), (2, "true", 2, "true", "false"), (2, "false", 2, "true", "true"),
         (1, "true", 1, "false", "false")]


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    """{product: its kernels' assembly}"""
    text = open(os.path.join(B.CSRC, "prod_w4.hpp")).read()
    assert text.count(WHICH) == 1
    runs = {}
    for second in ("false", "true"):
        d = tmp_path_factory.mktemp("asm")
        (d / "prod_w4.hpp").write_text(text.replace(WHICH, "constexpr bool second = %s;" % second))
        kernels = ["template __global__ void prod_w4_two_kernel<%s>(ProdPair, %s);" % (", ".join((str(t), *e)), ", ".join(e))
                   for t, vec, ot, vec1, add in FORMS
                   for e in [("Known<PlainEpi<%d>, %s, false>" % (t, vec), "Known<PlainEpi<%d>, %s, %s>" % (ot, vec1, add))]]
        (d / "two.hip").write_text(HEAD + "\n".join(kernels) + "\n}\n")
        runs[second] = subprocess.Popen([B.HIPCC] + B.FLAGS + ["-I" + B.CSRC, "-S", "--cuda-device-only", str(d / "two.hip"),
                                                              "-o", str(d / "two.s")], stderr=subprocess.DEVNULL), d / "two.s"
    assert [r.wait() for r, _ in runs.values()] == [0, 0]
    return {second: out.read_text() for second, (_, out) in runs.items()}


def kernels(text):
    return sorted(set(re.findall(r"^(_ZN2tg\w*prod_w4_two_\w+):", text, re.M)))


def at_barrier(name, queue):
    assert not any(q >= 2 for q in queue), "an operand's load may still be on its way behind this barrier"


@pytest.mark.parametrize("second", ["false", "true"])
def test_operands_have_landed_at_every_barrier(assembly, second):
    names = kernels(assembly[second])
    assert len(names) == len(FORMS)
    for name in names:
        assert follow(assembly[second], name, at_barrier, at_end) > 4, name


@pytest.mark.parametrize("second,wait", [("false", 1), ("true", 1), ("false", 32)])
def test_the_check_sees_waits_that_are_too_short(assembly, second, wait):
    """One operation more left in flight, at the K tiles' ends or behind the results."""
    text = assembly[second]
    assert "vmcnt(%d)" % wait in text
    with pytest.raises(AssertionError):
        for name in kernels(text):
            follow(text.replace("vmcnt(%d)" % wait, "vmcnt(%d)" % (wait + 1)), name, at_barrier, at_end)
