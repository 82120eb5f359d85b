"""dspark_append and rows that are not as dspark_pack writes them: a row that follows no row of its
request, begins no page and is not its request's first has no owner; it is not stored, and said so."""
import numpy as np
import pytest
import torch

from speculative_decoding_ragged_gb300 import _binding as bd
from test_gpu_append import Case

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_ragged_gb300 import build
    build.build()
    return bd.lib()


@gpu
@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("w,lengths,page", [([3, 4, 5, 2], [3, 17, 2, 30], 16), ([100, 90], [9, 70], 32)])
def test_rows_that_follow_none_are_flagged(lib, w, lengths, page, first):
    c = Case(3, w, lengths, 2, 1, 64, page, "bf16")
    want = c.want()
    b = first
    rows = np.flatnonzero(c.req == b)
    c.pos[rows[1:]] += 1                      # a gap after the request's first row
    got = c.run(None)
    assert got["status"] == bd.STATUS_BAD_ROWS
    for name in "kv":
        others = np.setdiff1d(np.arange(c.n), c.table[b])
        np.testing.assert_array_equal(got[name][others], want[name][others])


@gpu
def test_a_request_that_starts_late(lib):
    """Its first row is not position 0: nothing of its first page is stored; at a page's start it is."""
    c = Case(4, [4, 20], [1, 14], 2, 1, 64, 16, "f32")
    c.pos[c.req == 0] += 2
    got = c.run(None)
    assert got["status"] == bd.STATUS_BAD_ROWS
    p = c.table[0, 0]
    np.testing.assert_array_equal(got["k"][p], c.codes["k"][p])
    np.testing.assert_array_equal(got["ks"][p], c.scale["k"][p])
    c.pos[c.req == 0] -= 2
    assert c.run(None)["status"] == 0


@gpu
def test_padding_between_requests_is_no_fault(lib):
    c = Case(5, [3, 4, 2], [15, 3, 40], 2, 1, 64, 16, "bf16")
    c.req = np.insert(c.req, [3, 3, 7], -1).astype(np.int32)
    c.pos = np.insert(c.pos, [3, 3, 7], -1).astype(np.int32)
    c.proj = torch.cat([c.proj, c.proj[:3]])
    c.rows += 3
    got, want = c.run(None), c.want()
    assert got["status"] == 0
    np.testing.assert_array_equal(got["k"], want["k"])
