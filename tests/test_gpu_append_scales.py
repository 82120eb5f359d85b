"""dspark_append into blocks whose scale is no power of two (a cache filled elsewhere): the codes are
those of the exact quotients and products, ties and all. Compared bit for bit with 64 bits, which
tell a tie from its neighbours here: products and quotients of 24-bit numbers."""
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


def same(c):
    got, want = c.run(None), c.want()
    for name in ("k", "v", "ks", "vs"):
        np.testing.assert_array_equal(got[name], want[name], err_msg=name)
    assert got["status"] == 0
    return want


# windows inside a block and across two, prompts in teams, more rows than registers hold
SHAPES = [([3, 8], [5, 30], 2, 64, 16), ([20], [70], 3, 128, 32), ([100, 2], [9, 77], 2, 96, 64),
          ([70], [100], 4, 128, 128), ([5, 5], [3, 120], 1, 256, 128)]


def rows_by_block(c):
    for r, (b, i) in enumerate(zip(c.req, c.pos)):
        if b >= 0:
            t = int(c.lengths[b]) + int(i)
            if t // c.page == int(c.lengths[b]) // c.page and int(c.lengths[b]) % c.page:
                yield r, int(c.table[b, t // c.page])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_kept_scales_of_any_mantissa(lib, shape, dtype):
    w, lengths, heads, dim, page = shape
    c = Case(dim + page, w, lengths, heads, 1, dim, page, dtype, spread=0.0)
    rng = np.random.default_rng(1)
    for s in c.scale.values():                # above every fresh one: the old scale stays
        s[:] = np.exp2(rng.uniform(-5, -4, s.shape)).astype(np.float32)
    want = same(c)
    kept = [p for _, p in rows_by_block(c)]
    assert (want["ks"][kept] == c.scale["k"][kept]).all()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_quotients_beside_ties(lib, shape, dtype):
    """Elements whose quotients lie between two codes, some exactly, some off by the scale's last bit."""
    w, lengths, heads, dim, page = shape
    c = Case(dim + page + 1, w, lengths, heads, 1, dim, page, dtype, spread=0.0)
    rng = np.random.default_rng(2)
    ties = np.array([17, 19, 21, 23, 25, 27, 29, 31]) / 2.0      # midway between 4-bit numbers
    x = c.proj.double().numpy()
    for name, h0 in (("k", heads), ("v", 2 * heads)):
        c.scale[name][:] = np.float32(0.07)   # above every fresh one: it stays
        for r, p in rows_by_block(c):
            for h in range(heads):
                tie = rng.choice(ties, dim) * np.exp2(rng.integers(-4, 4, dim))
                x[r, h0 + h] = tie * float(c.scale[name][p, h]) * rng.choice([-1, 1], dim)
    c.proj = torch.as_tensor(x).to(c.dtype)
    same(c)


@gpu
@pytest.mark.parametrize("page", [16, 64])
def test_retained_codes_under_a_growing_scale_of_any_mantissa(lib, page):
    c = Case(7, [2, 40], [13, page + 9], 3, 1, 128, page, "f32", spread=0.0)
    rng = np.random.default_rng(3)
    # old scales that put codes beside ties of the new, larger one
    for s in c.scale.values():
        s[:] = (np.float32(1.0) / rng.choice([3, 5, 7, 9, 11, 13], s.shape) * 17 / 2 ** 14).astype(np.float32)
    want = same(c)
    p = c.table[1, 1]
    assert (want["ks"][p] > c.scale["k"][p]).all()
