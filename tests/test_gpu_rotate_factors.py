"""The factors of dspark_rotate on their own: a head of (1, 0) pairs comes out as (cos, sin). Far
positions included, they are within the angle's rounding and the sine's own of 64 bits: the angle is
taken from the nearest quarter turn, so its fp32 rounding is 2^-27 half turns at most (2.4e-8 rad with
what is cut off before), and the sine and cosine are within one last place, 2^-24 under 1."""
import numpy as np
import pytest
import torch

import cache_ref as ref
from speculative_decoding_ragged_gb300 import _binding as bd

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_ragged_gb300 import build
    build.build()
    return bd.lib()


@gpu
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_factors(lib, interleaved, inverse):
    rng = np.random.default_rng(5)
    rows, dim = 4096, 128
    turns = rng.integers(0, 2 ** 63, dim // 2, dtype=np.uint64) * 2
    pos = rng.integers(-2 ** 31, 2 ** 31, rows).astype(np.int32)
    pos[:4] = 0, 1, -1, 2 ** 31 - 1
    x = np.zeros((rows, 1, dim))
    if interleaved:
        x[..., 0::2] = 1.0
    else:
        x[..., :dim // 2] = 1.0
    dev = torch.device("cuda:0")
    y = torch.empty(rows, 1, dim, device=dev)
    rope = bd.Rope(torch.as_tensor(turns.view(np.int64)).to(dev), 1.0, interleaved)
    bd.dspark_rotate(torch.as_tensor(x).float().to(dev), y, torch.as_tensor(pos).to(dev), rope, inverse=inverse)
    err = np.abs(y.double().cpu().numpy() - ref.rotate(x, pos, turns, 1.0, interleaved, inverse))
    assert err.max() <= 2.4e-8 + 2.0 ** -24, err.max()
