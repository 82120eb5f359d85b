"""dspark_attend_shared's groups: numbers that are no requests, whatever their size."""
import numpy as np
import pytest
import torch

from speculative_decoding_ragged_gb300 import _binding as bd
from test_gpu_attend_shared import Shared

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_ragged_gb300 import build
    build.build()
    return bd.lib()


def alone(c):
    """dspark_attend's results for the same call."""
    dev = torch.device("cuda:0")
    t = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(dev)         # noqa: E731
    cache = bd.PagedCache(t(c.codes["k"]), t(c.codes["v"]), t(c.scale["k"]), t(c.scale["v"]), t(c.table))
    q = torch.as_tensor(c.q).to(torch.bfloat16).to(dev)
    out = torch.full_like(q, 5.0)
    ws = torch.zeros(bd.dspark_attend_workspace_bytes(c.heads, c.dim), dtype=torch.uint8, device=dev)
    bd.dspark_attend(cache, q, out, t(c.cu), t(c.lengths), ws)
    return out.double().cpu().numpy()


def mixed(seed, w=None, more=70):
    """Groups of 3, 2 and `more` requests; enough tiles are saved where a few of the last are left out."""
    w = [2, 3, 1, 4, 2] + [1] * more if w is None else w
    return Shared(seed, w, [30, 5, 200, 64, 0] + [i % 5 for i in range(more)],
                  [(3, 160), (2, 320), (more, 128 * 48)], 2, 4, 128, 16, heavy=False)


@gpu
@pytest.mark.parametrize("numbers", [[2000000000, -2000000000], [-(1 << 31), (1 << 31) - 1], [0, (1 << 31) - 1],
                                     [(1 << 31) - 1, -(1 << 31)], [70, -(1 << 31) + 60, 75, 80], [1 << 30, 1 << 30]])
def test_numbers_that_are_no_requests(lib, numbers):
    """Whatever they are, differences that pass 32 bits too: every request attends alone."""
    c = mixed(21)
    c.group_cu = np.asarray(numbers, np.int32)
    c.prefix = np.full(len(numbers) - 1, 128, np.int32)
    out, _ = c.hold()
    np.testing.assert_array_equal(out, alone(c))
