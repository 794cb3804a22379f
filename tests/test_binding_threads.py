"""The binding's part in C++ towards the interpreter (CPU only): errors that
Python code raises below it."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

fast = pytest.importorskip("tiled_dense_gemm_tile_amd._tensors")


class Handler(TorchDispatchMode):
    """torch's operators answered by a Python function."""
    def __init__(self, answer):
        super().__init__()
        self.answer = answer

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        return self.answer()


def test_errors_of_python_code_below_an_allocation():
    """They come out as they are, and leave the binding usable."""
    def fails():
        raise KeyError("mine")

    with Handler(fails), pytest.raises(KeyError, match="mine"):
        fast.empty((2, 3), torch.float32, 0)
    some = torch.zeros(2, 3)
    with Handler(lambda: some):
        assert fast.empty((2, 3), torch.float32, 0) is some
    assert fast.matrix(some, (2, 3), (torch.float32,), -1) == (some.data_ptr(), 3)
