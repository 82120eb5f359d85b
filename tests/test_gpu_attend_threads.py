"""dspark_attend called first from several host threads at once, each on its own stream: every thread
makes the kernels' set-up for itself, and gets the result of a call alone."""
import threading

import numpy as np
import pytest
import torch

from speculative_decoding_ragged_gb300 import _binding as bd
from test_gpu_attend import Case

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_ragged_gb300 import build
    build.build()
    return bd.lib()


@gpu
@pytest.mark.parametrize("w,dim", [([3, 1], 128), ([90, 40], 128), ([8], 64), ([150], 64)])
def test_first_calls_from_many_threads(lib, w, dim):
    c = Case(11, w, [300] * len(w), 2, 4, dim, 32)
    got = [None] * 6

    def work(i):
        torch.cuda.set_device(0)
        with torch.cuda.stream(torch.cuda.Stream()):
            got[i] = c.run(torch.bfloat16)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(got))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    _, want, lse, _ = c.run(torch.bfloat16)
    for _, out, ls, st in got:
        assert st == 0
        np.testing.assert_array_equal(out, want)
        np.testing.assert_array_equal(ls, lse)
