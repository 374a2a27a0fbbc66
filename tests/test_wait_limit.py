"""The bounded waits of the block-wise scan: a barrier that nobody arrives at ends the wait at its
limit, for a whole warp at once, and the kernel frees what it holds, ends and reports the timeout."""

import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from sparse_memory_linear_b200.build import NVCC_FLAGS, _nvcc
    out = str(tmp_path_factory.mktemp("wait") / "libwait.so")
    subprocess.run([_nvcc(), *NVCC_FLAGS, "-o", out, os.path.join(HERE, "mbar_wait_limit.cu")],
                   check=True)
    return ctypes.CDLL(out)


def test_the_waits_compile_on_their_own(lib):
    assert lib.run_wait


@pytest.mark.gpu
def test_waits_end_at_their_limit(lib):
    import torch
    assert torch.cuda.is_available()
    for arrive, ok, word in ((1, 1, 0), (0, 0, 2), (1, 1, 0)):
        out, status = (ctypes.c_int * 128)(), ctypes.c_uint(99)
        assert lib.run_wait(arrive, out, ctypes.byref(status)) == 0
        assert status.value == word
        for w in range(4):
            lanes = list(out)[32 * w:32 * w + 32]
            assert [x & 1 for x in lanes] == [ok] * 32   # a warp goes on or gives up as one
            assert sum(x >> 1 for x in lanes) == 1       # and elects one lane behind it
