"""The history that the decode loop gives dspark_adjust: the shared prompt's tokens, the first anchor,
then what was committed. The expectation is built from those, not from the loop's buffers."""
import numpy as np
import pytest
import torch

from speculative_decoding_ragged_gb300.decode import DecodeLoop

from gpu_util import device

pytestmark = pytest.mark.gpu


def ints(t):
    return t.cpu().numpy().astype(np.int64)


@pytest.mark.parametrize("prompt", [0, 48])
def test_the_prompt_and_the_first_anchor_count(prompt):
    """repetition: tokens of the prompt, the anchor and the answer; presence and frequency: the anchor and
    the answer. 61 tokens, so that most are met at once."""
    B, V = 5, 61
    loop = DecodeLoop(B, 4, V, prompt=prompt, repetition=1.3, presence=0.5, frequency=0.7, max_len=64,
                      seed=3, device=device())
    given = ints(loop.prompt)
    assert len(given) == prompt
    answers = [[int(a)] for a in ints(loop.anchor)]
    for _ in range(6):
        tokens, conf = loop.draft()
        assert (ints(tokens)[:, 0] == [a[-1] for a in answers]).all()       # the history's last is the anchor
        loop.step.schedule_pack(conf, tokens)
        logits = loop.target()
        raw = logits.double().cpu().numpy()
        loop.step.adjust(logits, tokens, loop.how)
        got, cu = logits.double().cpu().numpy(), ints(loop.step.cu)
        for b in range(B):
            for i in range(cu[b + 1] - cu[b]):
                x = raw[cu[b] + i]
                uses = np.bincount(np.concatenate([answers[b], ints(tokens)[b, 1:i + 1]]).astype(int), minlength=V)
                seen = (uses > 0) | (np.bincount(given, minlength=V) > 0)
                x = np.where(seen, np.where(x > 0, x / 1.3, x * 1.3), x)
                x = x - np.where(uses > 0, 0.7 * uses + 0.5, 0.0)
                # the penalties' and three results' roundings to fp32, one to bf16
                err = np.abs(got[cu[b] + i] - x)
                assert (err <= 2.0 ** -8 * np.abs(x) + 2.0 ** -20 * (np.abs(x) + 20)).all()
        loop.step.verify_scatter(logits, tokens)
        L, committed = ints(loop.step.accept_len), ints(loop.step.committed)
        for b in range(B):
            answers[b] += committed[b, :L[b]].tolist()
        loop.advance()
    n, kept = ints(loop.step.out_len), ints(loop.step.out_tokens)
    for b in range(B):
        assert kept[b, :n[b]].tolist() == given.tolist() + answers[b]
    assert int(loop.step.status.item()) == 0 and int(loop.attention.status.item()) == 0


def test_as_long_as_the_pages_hold():
    """A loop that commits up to its longest context: no history overflows."""
    loop = DecodeLoop(3, 4, 128, prompt=32, frequency=0.2, max_len=40, seed=1, device=device())
    while int(loop.lengths.max()) + 4 <= 32 + 40:
        loop.run()
    assert (ints(loop.step.out_len) == ints(loop.lengths) + 1).all()
    assert int(loop.step.status.item()) == 0 and int(loop.attention.status.item()) == 0
