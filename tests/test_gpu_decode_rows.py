"""Rows past the packed ones. dspark_pack leaves the rows past its tier as they were, so a buffer of
capacity rows holds an earlier step's owners there. They must not reach the cache: its values are
compared bit for bit with the definition's over the packed rows alone."""
import numpy as np
import pytest
import torch

import cache_ref as ref
from speculative_decoding_ragged_gb300 import _binding as bd
from speculative_decoding_ragged_gb300.decode import CachedAttention, DecodeLoop, packed_owners

from gpu_util import device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return device()


def values(cache):
    return cache.v.view(torch.uint8).cpu().numpy(), cache.v_scale.cpu().numpy()


@pytest.mark.parametrize("dim,page,seed", [(64, 16, 1), (64, 32, 2), (128, 16, 3), (128, 32, 4)])
def test_a_loop_stores_the_packed_rows_only(dev, dim, page, seed):
    loop = DecodeLoop(5, 4, 512, dim=dim, page=page, seed=seed, device=dev)
    att, step = loop.attention, loop.step
    table = att.cache.table.cpu().numpy()
    tiers = set()
    for _ in range(12):
        codes, scale = values(att.cache)
        lengths = loop.lengths.cpu().numpy()
        tokens, conf = loop.draft()
        step.schedule_pack(conf, tokens)
        logits = loop.target()
        M = int(step.cu[-1])
        tiers.add(int(step.meta[1]))
        v = loop.project(loop.emb[step.packed_ids.clamp(0, loop.V - 1).long()])[2].double().cpu().numpy()
        ref.append(codes, scale, v[:M], step.row_req.cpu().numpy()[:M], step.row_pos.cpu().numpy()[:M],
                   lengths, table)
        got, got_scale = values(att.cache)
        np.testing.assert_array_equal(got_scale, scale)
        np.testing.assert_array_equal(got, codes)
        step.verify_scatter(logits, tokens)
        loop.advance()
    assert int(att.status.item()) == 0
    assert min(tiers) < step.packed_cap       # some steps left rows past their tier


@pytest.mark.parametrize("rows,B", [(29, 5), (300, 3)])
def test_a_layer_ignores_rows_past_the_packed_ones(dev, rows, B):
    rng = np.random.default_rng(rows)
    put = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(dev)     # noqa: E731
    w = rng.multinomial(rows, np.ones(B) / B)
    cu = np.concatenate([[0], np.cumsum(w)]).astype(np.int32)
    req, pos = np.repeat(np.arange(B), w), np.concatenate([np.arange(x) for x in w])
    lengths = rng.integers(0, 40, B).astype(np.int32)
    more = 13
    q, k, v = (torch.randn(rows + more, h, 64, device=dev).bfloat16() for h in (8, 2, 2))
    blocks = (rows + 60) // 16 + 1
    table = put(rng.permutation(B * blocks).astype(np.int32).reshape(B, blocks))
    outs = []
    for stale in (False, True):
        att = CachedAttention(rows + more, 8, 2, 64, table, B * blocks, 16, bd.Rope.make(64, device=dev))
        r = np.concatenate([req, req[:more] if stale else -np.ones(more)]).astype(np.int32)
        p = np.concatenate([pos, pos[:more] if stale else -np.ones(more)]).astype(np.int32)
        out = att.run(q, k, v, put(r), put(p), put(cu), put(lengths))
        outs.append([out[:rows].clone(), att.cache.k.view(torch.uint8), att.cache.v.view(torch.uint8),
                     att.cache.k_scale, att.cache.v_scale, att.status])
        owners = packed_owners(put(r), put(cu))
        assert owners.tolist() == req.tolist() + [-1] * more
        again = att.run(q, k, v, owners, put(p), put(cu), put(lengths), owned=True)
        assert torch.equal(again[:rows], outs[-1][0])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
