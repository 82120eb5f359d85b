"""dspark_adjust: a bias of -inf bans its token whatever the logit is, and rows that are left without a
token through verify, greedy and stochastic."""
import numpy as np
import pytest
import torch

from speculative_decoding_ragged_gb300 import _binding as bd
from speculative_decoding_ragged_gb300.decode import DecodeLoop

from gpu_util import device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_a_bias_of_minus_infinity_bans(dtype, in_place, masked):
    """Banned: every second token of a request's list, whose logits are infinities, NaN and ordinary ones;
    the others' finite biases follow the formula."""
    dev = device()
    V, B, gamma, n = 2051, 2, 3, 40
    rng = np.random.default_rng(7)
    ids = np.stack([rng.permutation(V)[:n] for _ in range(B)]).astype(np.int32)
    x = rng.standard_normal((B * gamma, V)).astype(np.float32)
    for b in range(B):
        for i in range(gamma):
            row = x[b * gamma + i]
            row[ids[b, 0:16]] = np.inf
            row[ids[b, 16:24]] = np.nan
            row[ids[b, 24:28]] = -np.inf
    x = torch.as_tensor(x).to(dev, dtype)
    values = np.where(np.arange(n) % 2 == 0, -np.inf, 1.5).astype(np.float32)
    put = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(dev)       # noqa: E731
    # penalties too: the history has half of the banned tokens
    how = bd.Adjustments(history=put(ids[:, :20]), history_len=put(np.full(B, 20, np.int32)),
                         repetition=put(np.full(B, 1.25, np.float32)), frequency=put(np.full(B, 0.5, np.float32)),
                         bias_tokens=put(ids), bias_values=put(np.tile(values, (B, 1))),
                         bias_len=put(np.full(B, n, np.int32)),
                         mask=put(np.full((1, -(-V // 32)), -1, np.int32)) if masked else None,
                         mask_row=put(np.zeros(B * gamma, np.int32)) if masked else None)
    out = x.clone()
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    bd.dspark_adjust(out if in_place else x, out, put(np.zeros((B, gamma), np.int32)), how, status=status)
    got, given = out.double().cpu().numpy(), x.double().cpu().numpy()
    for b in range(B):
        rows = slice(b * gamma, (b + 1) * gamma)
        assert np.isneginf(got[rows][:, ids[b, ::2]]).all()
        rest = ids[b, 21::2]                     # in no history: the bias alone
        want = given[rows][:, rest] + 1.5
        assert (np.isnan(got[rows][:, rest]) == np.isnan(want)).all()
        fine = np.isfinite(want)
        # one sum in fp32 and one rounding to the type
        err = np.abs(got[rows][:, rest][fine] - want[fine])
        assert (err <= (2.0 ** -24 + torch.finfo(dtype).eps / 2) * (np.abs(want[fine]) + 4)).all()
    assert int(status.item()) == 0


@pytest.mark.parametrize("stochastic", [False, True])
@pytest.mark.parametrize("V", [64, 700])
def test_rows_without_a_token(stochastic, V):
    """A grammar that allows nothing is flagged, and what verify commits is a token of the vocabulary all
    the same: the first one where it is greedy."""
    dev = device()
    loop = DecodeLoop(4, 3, V, mask=torch.zeros(-(-V // 32), dtype=torch.int32, device=dev), device=dev)
    step = loop.step
    step.stochastic = stochastic
    step.workspace = torch.zeros(bd.dspark_verify_workspace_bytes(4, 3, V, stochastic), dtype=torch.uint8, device=dev)
    draft = torch.zeros(4, 2, V, dtype=torch.bfloat16, device=dev) if stochastic else None
    for k in range(3):
        tokens, conf = loop.draft()
        step.schedule_pack(conf, tokens)
        logits = loop.target()
        step.adjust(logits, tokens, loop.how)
        M = int(step.cu[-1])
        assert bool(torch.isneginf(logits[:M]).all())
        step.verify_scatter(logits, tokens, draft, seed=5, step=k)
        L, committed = step.accept_len.tolist(), step.committed.tolist()
        for n, row in zip(L, committed):
            assert 1 <= n <= 3 and all(0 <= t < V for t in row[:n]) and row[n:] == [-1] * (3 - n)
            if not stochastic:
                assert row[:n] == [0] * n
        loop.advance()
    assert int(step.status.item()) == bd.STATUS_NO_TOKEN
