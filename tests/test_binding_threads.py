"""The binding's part in C++ towards the interpreter (CPU only): errors that
Python code raises below it, and other threads while it allocates."""
import sys
import threading
import time

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


def test_allocations_let_other_threads_run():
    """Results are allocated without the interpreter's lock.  With a switch interval that never ends, another thread
    runs between the call and the operator's Python handler only if the binding gives the lock up there; of many
    calls some meet that thread ready to run."""
    ran, stop, seen = [0], [], []

    def work():
        while not stop:
            ran[0] += 1
            time.sleep(0)

    some = torch.zeros(2, 3)

    def answer():
        seen.append(ran[0])
        return some

    every = sys.getswitchinterval()
    sys.setswitchinterval(1000)
    t = threading.Thread(target=work)
    t.start()
    try:
        with Handler(answer):
            for _ in range(200000):
                before = ran[0]
                fast.empty((2, 3), torch.float32, 0)
                if seen[-1] != before:
                    break
                time.sleep(0)
        assert seen[-1] != before
    finally:
        stop.append(True)
        sys.setswitchinterval(every)
        t.join()
