"""The build where the binding's part in C++ cannot be made (CPU only): the
library is built all the same, and no older binding is left beside it."""
import os
import shutil
import sys

import pytest

from tiled_dense_gemm_tile_amd import build as B

pytestmark = pytest.mark.skipif(shutil.which(B.HIPCC) is None and not os.path.exists(B.HIPCC),
                                reason="hipcc not available")

UNIT = r"""
#include <hip/hip_runtime.h>
__global__ void twice(const float *x, float *y) { y[threadIdx.x] = 2.0f * x[threadIdx.x]; }
extern "C" int answer() { return 42; }
"""


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A library of one unit, built into a directory of its own."""
    src = tmp_path / "one.hip"
    src.write_text(UNIT)
    monkeypatch.setattr(B, "sources", lambda: [str(src)])
    for name, path in (("OUT", "lib.so"), ("BINDING", "_tensors.so"), ("OBJDIR", "obj")):
        monkeypatch.setattr(B, name, str(tmp_path / path))
    (tmp_path / "_tensors.so").write_text("of an older build")
    return tmp_path


def without_torch(m):
    m.setitem(sys.modules, "torch", None)


def without_compiler(m):
    m.setenv("PATH", "/nowhere")


def without_sources(m):
    m.setattr(B, "CSRC", "/nowhere")


@pytest.mark.parametrize("lack", [without_torch, without_compiler, without_sources])
def test_library_without_the_binding(small, lack, monkeypatch, capsys):
    lack(monkeypatch)
    assert B.build() == str(small / "lib.so")
    assert (small / "lib.so").exists() and not (small / "_tensors.so").exists()
    assert "_tensors.so" in capsys.readouterr().err


def test_library_with_the_binding(small):
    B.build(verbose=False)
    assert (small / "lib.so").exists() and (small / "_tensors.so").stat().st_size > 10000
