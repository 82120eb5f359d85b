"""dspark_attend_shared's groups: numbers that are no requests, whatever their size; first members that
have no rows, or fewer tokens than the prefix, and table rows of which nothing is said; members that do
not count; far more groups than requests; every kernel that the prefixes and the own tokens can take."""
import numpy as np
import pytest
import torch

import forms_ref
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


def saved(c):
    """Tiles of 128 tokens and a head that are not read again, over the members that have the prefix and rows."""
    n = 0
    for g, p in enumerate(c.prefix // c.page * c.page):
        b = np.arange(c.group_cu[g], c.group_cu[g + 1])
        joins = ((c.lengths[b] >= p) & (np.diff(c.cu)[b] > 0)).sum()
        n += max(int(joins) - 1, 0) * -(-int(p) // 128) * c.heads
    return n


def mixed(seed, w=None, more=70):
    """Groups of 3, 2 and `more` requests; enough tiles are saved where a few of the last are left out."""
    w = [2, 3, 1, 4, 2] + [1] * more if w is None else w
    return Shared(seed, w, [30, 5, 200, 64, 0] + [i % 5 for i in range(more)],
                  [(3, 160), (2, 320), (more, 128 * 48)], 2, 4, 128, 16, heavy=False)


def other_pages(c, b, at):
    """Request b's entries from `at` on are other pages of the cache."""
    c.table[b, at:] = np.random.default_rng(b).integers(0, c.n, c.table.shape[1] - at)


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


@gpu
@pytest.mark.parametrize("what", ["short", "empty", "retired", "several", "wrong rows"])
def test_first_members_without_the_prefix(lib, what):
    """A group's pages are read by a member that has them."""
    w = [2, 3, 1, 4, 2] + [1] * 70
    if what in ("empty", "retired"):
        w[0] = w[3] = w[5] = 0
    if what == "several":
        w[6] = w[7] = 0
    c = mixed(22, w)
    if what == "short":                          # fewer tokens than the prefix: other pages behind them
        c.lengths[[0, 3, 5]] = 100, 1, 40
        for b, at in ((0, 7), (3, 1), (5, 3)):
            other_pages(c, b, at)
    elif what == "empty":                        # slots without tokens or pages
        c.lengths[[0, 3, 5]] = 0
        c.table[[0, 3, 5]] = -7
    elif what == "retired":                      # slots whose lengths are as they were, their pages others'
        for b in (0, 3, 5):
            other_pages(c, b, 0)
    elif what == "several":
        c.lengths[5:8] = 0, 40, 100000
        other_pages(c, 5, 1)
        c.table[6:8] = c.n
    else:                                        # a first member whose rows run backwards
        c.cu[5:7] = [12, 8]                      # request 5 has none; request 6 has its row and 5's and request 4's
        c.w[5], c.w[6] = 0, 5
        other_pages(c, 5, 0)
        assert saved(c) >= 6000
        q, out, lse, st = c.go(torch.bfloat16)
        assert st & bd.STATUS_BAD_ROWS
        want = forms_ref.attend(c, q, c.dim ** -0.5, lambda b, pos: np.arange(pos + 1))[0]
        np.testing.assert_allclose(out[14:82], want[14:82], atol=0.02, rtol=0.02)
        return
    assert saved(c) >= 6000
    out, lse = c.hold()
    assert not np.array_equal(out, alone(c))     # prefixes were computed apart


@gpu
def test_first_members_among_many(lib):
    """More requests than threads plan them; the first that has the prefix comes late."""
    w = [0] * 990 + [1] * 10 + [0] * 100 + [1] * 400 + [3, 0]
    B = len(w)
    c = Shared(23, w, [i % 3 for i in range(B)], [(1000, 64), (500, 1040), (2, 32)], 2, 2, 64, 16, heavy=False)
    for b in np.flatnonzero(np.asarray(w) == 0):
        c.lengths[b] = (0, 50, 100000)[b % 3]
        c.table[b] = -7 if b % 2 else (b * 31 + np.arange(c.table.shape[1])) % c.n
    assert saved(c) >= 6000
    out, lse = c.hold()
    assert not np.array_equal(out, alone(c))


@gpu
def test_a_prefix_that_no_member_has(lib):
    """Nobody sees its pages: nothing is said of them, whatever the table holds."""
    c = mixed(24)
    c.lengths[:3] = 100, 0, 30
    for b, at in ((0, 7), (1, 1), (2, 2)):
        c.table[b, at:] = -7
    c.lengths[3:5] = 319, 0                      # a token too few
    c.table[4, 1:] = c.n
    c.hold()


@gpu
def test_members_without_the_prefix_do_not_count(lib):
    """Whether it pays is a matter of the members that join."""
    c = mixed(25)
    c.lengths[7:65] = 100
    assert 0 < saved(c) < 6000
    out, _ = c.hold()
    np.testing.assert_array_equal(out, alone(c))


@gpu
def test_far_more_groups_than_requests(lib):
    """Empty groups, so many that the prefixes' line is longer than a call can cut: as dspark_attend."""
    c = mixed(26)
    n = 10_000_000
    tiles = -(-c.table.shape[1] * c.page // 128)
    assert n * c.heads * (tiles + 4) > 1 << 30
    c.group_cu = np.concatenate([np.zeros(n, np.int32), c.group_cu])
    c.prefix = np.concatenate([np.full(n, 128, np.int32), c.prefix])
    out, _ = c.hold()
    np.testing.assert_array_equal(out, alone(c))
    c.group_cu, c.prefix = c.group_cu[n - 100:], c.prefix[n - 100:]         # a hundred of them
    out, _ = c.hold()
    assert not np.array_equal(out, alone(c))


def unit_rows(rows, group, n):
    """The kernel that n requests (or groups) of together `rows` rows and a cache head's `group` query heads take:
    the narrow one of 8, 16 or 32 rows a unit, the wide one of 128."""
    return next((r for r in (8, 16, 32) if rows * group <= r * n), 128)


def many(n, size, w, group, heads, dim, page, prefix, seed):
    """n groups of about `size` requests with windows of about w."""
    rng = np.random.default_rng(seed)
    sizes = size + rng.integers(-1, 2, n)
    ws = np.maximum(w + rng.integers(-1, 1, sizes.sum()) * (rng.random(sizes.sum()) < 0.3), 1)
    own = rng.integers(0, 40, sizes.sum()) * (rng.random(sizes.sum()) < 0.5)
    return Shared(seed, ws, own, [(int(s), prefix) for s in sizes], heads, group, dim, page, heavy=False)


# n, size, w, group, heads, dim, page, prefix; the rows of a prefix's units and of an own unit
KERNELS = [((30, 6, 1, 1, 8, 128, 16, 720), 8, 8), ((30, 6, 2, 1, 8, 128, 32, 704), 16, 8),
           ((30, 6, 2, 2, 8, 128, 16, 720), 32, 8), ((32, 6, 1, 1, 8, 64, 16, 656), 8, 8),
           ((32, 6, 2, 1, 8, 64, 64, 704), 16, 8), ((40, 5, 3, 2, 8, 64, 16, 592), 32, 8),
           ((160, 6, 1, 1, 8, 128, 64, 128), 8, 8), ((160, 6, 2, 2, 8, 64, 16, 112), 32, 8),
           ((260, 3, 1, 2, 8, 64, 32, 192), 8, 8),
           ((2, 10, 8, 3, 2, 128, 64, 21760), 128, 32), ((2, 16, 12, 4, 2, 64, 64, 13952), 128, 128),
           ((3, 12, 6, 4, 2, 64, 16, 13040), 128, 32)]


@gpu
@pytest.mark.parametrize("shape,prefix_rows,own_rows", KERNELS)
def test_every_kernel(lib, shape, prefix_rows, own_rows):
    c = many(*shape, seed=sum(shape))
    assert unit_rows(c.rows, shape[3], len(c.prefix)) == prefix_rows
    assert unit_rows(c.rows, shape[3], len(c.lengths)) == own_rows
    assert saved(c) >= 6000
    out, _ = c.hold()
    assert not np.array_equal(out, alone(c))
    np.testing.assert_array_equal(c.go(torch.bfloat16, lse=False, fill=0xFF)[1], out)
