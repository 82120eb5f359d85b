"""The decode loop with the target's other operators: a window with sinks, a prompt shared by all
requests, adjusted logits; whole steps of them captured and replayed, with other workspaces and on
another stream; the layer's refusals."""
import numpy as np
import pytest
import torch

import forms_ref
from speculative_decoding_ragged_gb300 import _binding as bd
from speculative_decoding_ragged_gb300.decode import CachedAttention, DecodeLoop

from gpu_util import device

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return device()


def test_the_layer_refuses():
    table = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="need a window"):
        CachedAttention(1, 1, 1, 64, table, 1, 16, sinks=4)
    with pytest.raises(ValueError, match="no window"):
        CachedAttention(1, 1, 1, 64, table, 1, 16, window=4, shared=(None, None))


def ints(t):
    return t.cpu().numpy().astype(np.int64)


class Held:
    """A layer's cache as forms_ref takes it."""

    def __init__(self, att, cu, lengths):
        c = att.cache
        self.n, self.heads, self.page, self.dim, self.hq = c.n_pages, c.heads, c.page, c.dim, att.out.shape[1]
        self.codes = {"k": c.k.view(torch.uint8).cpu().numpy(), "v": c.v.view(torch.uint8).cpu().numpy()}
        self.scale = {"k": c.k_scale.view(self.n, -1).cpu().numpy(), "v": c.v_scale.view(self.n, -1).cpu().numpy()}
        self.table, self.cu, self.lengths = c.table.cpu().numpy(), cu, lengths


def attention_holds(att, cu, lengths, seen, joined=False):
    M = int(cu[-1])
    out = att.out[:M].double().cpu().numpy()
    forms_ref.check(Held(att, cu, lengths), torch.bfloat16, att.turned[:M].double().cpu().numpy(), out, None, seen,
                    joined=joined)


@gpu
@pytest.mark.parametrize("dim,page,window,sinks", [(64, 16, 9, 2), (128, 32, 20, 33)])
def test_sinks(dev, dim, page, window, sinks):
    loop = DecodeLoop(5, 4, 512, dim=dim, page=page, window=window, sinks=sinks, seed=dim, device=dev)

    def seen(b, pos):
        t = np.arange(pos + 1)
        return t[(t > pos - window) | (t < sinks)]

    for _ in range(window + sinks + 2):          # a token a step at least
        before = ints(loop.lengths)
        tokens, conf = loop.draft()
        loop.step.schedule_pack(conf, tokens)
        logits = loop.target()
        attention_holds(loop.attention, ints(loop.step.cu), before, seen)
        loop.step.verify_scatter(logits, tokens)
        loop.advance()
    assert int(loop.lengths.min()) > window + sinks
    assert int(loop.step.status.item()) == 0 and int(loop.attention.status.item()) == 0


@gpu
@pytest.mark.parametrize("B,prompt", [(5, 48), (64, 6144)])      # attended alone; computed apart
def test_shared_prompt(dev, B, prompt):
    loop = DecodeLoop(B, 4, 512, page=16, prompt=prompt, max_len=64, seed=B, device=dev)
    for _ in range(3):
        before = ints(loop.lengths)
        tokens, conf = loop.draft()
        loop.step.schedule_pack(conf, tokens)
        logits = loop.target()
        attention_holds(loop.attention, ints(loop.step.cu), before, lambda b, pos: np.arange(pos + 1), joined=True)
        loop.step.verify_scatter(logits, tokens)
        loop.advance()
    assert (ints(loop.step.out_len) == ints(loop.lengths) - prompt).all()
    assert int(loop.step.status.item()) == 0 and int(loop.attention.status.item()) == 0


@gpu
@pytest.mark.parametrize("stochastic", [False, True])
def test_adjusted_logits_are_what_verify_sees(dev, stochastic):
    """A grammar of few tokens and heavy penalties: what is committed is allowed, and greedily the best
    of the adjusted rows."""
    V = 515
    rng = np.random.default_rng(3)
    allowed = rng.random(V) < 0.1
    words = np.zeros(-(-V // 32) * 32, bool)
    words[:V] = allowed
    mask = torch.as_tensor(np.packbits(words, bitorder="little").view(np.int32).copy()).to(dev)
    loop = DecodeLoop(6, 4, V, repetition=1.3, presence=0.5, frequency=0.7, mask=mask, seed=5, device=dev)
    step = loop.step
    step.stochastic = stochastic
    ws = bd.dspark_verify_workspace_bytes(6, 4, V, stochastic)
    step.workspace = torch.zeros(ws, dtype=torch.uint8, device=dev)
    draft = torch.zeros(6, 3, V, dtype=torch.bfloat16, device=dev)
    for k in range(10):
        tokens, conf = loop.draft()
        step.schedule_pack(conf, tokens)
        logits = loop.target()
        raw = logits.float().cpu().numpy()
        n, history = ints(step.out_len), ints(step.out_tokens)
        step.adjust(logits, tokens, loop.how)
        M, cu = int(step.cu[-1]), ints(step.cu)
        got = logits.float().cpu().numpy()
        for b in range(6):
            for i in range(cu[b + 1] - cu[b]):
                x = raw[cu[b] + i].astype(np.float64)
                uses = np.bincount(np.concatenate([history[b, :n[b]], ints(tokens)[b, 1:i + 1]]), minlength=V)
                x = np.where(uses > 0, np.where(x > 0, x / 1.3, x * 1.3), x)
                x = x - np.where(uses > 0, 0.7 * uses + 0.5, 0.0)
                x[~allowed] = -np.inf
                y = got[cu[b] + i]
                assert np.isneginf(y[~allowed]).all()
                # three roundings to fp32 (and of the penalties given), one to bf16
                err = np.abs(y[allowed] - x[allowed])
                assert (err <= 2.0 ** -8 * np.abs(x[allowed]) + 2.0 ** -20 * (np.abs(x[allowed]) + 20)).all()
        assert np.array_equal(got[M:], raw[M:])                 # rows of no request
        step.verify_scatter(logits, tokens, draft if stochastic else None, seed=7, step=k)
        L, committed = ints(step.accept_len), ints(step.committed)
        best = got.argmax(-1)
        for b in range(6):
            last = committed[b, L[b] - 1]
            assert allowed[last]
            if not stochastic:
                assert (committed[b, :L[b]] == best[cu[b]:cu[b] + L[b]]).all()
        loop.advance()
    assert int(step.status.item()) == 0


@gpu
def test_a_row_without_tokens_is_flagged(dev):
    loop = DecodeLoop(2, 3, 64, mask=torch.zeros(2, dtype=torch.int32, device=dev), device=dev)
    loop.run()
    assert int(loop.step.status.item()) == bd.STATUS_NO_TOKEN
    assert ((ints(loop.step.committed) >= -1) & (ints(loop.step.committed) < 64)).all()


def whole_step(loop, tokens, conf, logits_in):
    """The calls of a step over fixed buffers: pack, the layer, the logits (a product of torch's in
    between is left out: they are given), adjust, verify."""
    s, att = loop.step, loop.attention
    x = loop.emb[s.packed_ids.clamp(0, loop.V - 1).long()]
    q, k, v = loop.project(x)
    out = torch.empty_like(logits_in)
    calls = [s.schedule_pack(conf, tokens, prepare=True)]
    calls += att.prepare(q, k, v, s.row_req, s.row_pos, s.cu, loop.lengths)
    calls += [s.adjust(logits_in, tokens, loop.how, out=out, prepare=True),
              s.verify_scatter(out, tokens, prepare=True)]
    return calls, out, (q, k, v)


@gpu
@pytest.mark.parametrize("more", [dict(window=30, sinks=5), dict(prompt=6144)])
def test_graph_replays_eager_steps(dev, more):
    """One captured step (attention, adjustments, verify) replayed twice, as two eager ones, on another
    stream than the eager ones."""
    def make():
        loop = DecodeLoop(64, 4, 600, repetition=1.2, frequency=0.3, max_len=96, seed=9, device=dev, **more)
        tokens, conf = loop.draft()
        loop.step.schedule_pack(conf, tokens)
        g = torch.Generator(device=dev).manual_seed(1)
        logits = torch.randn(loop.step.packed_cap, 600, generator=g, device=dev).bfloat16()
        return loop, tokens, conf, logits

    def state(loop, out):
        att, s = loop.attention, loop.step
        return [t.clone() for t in (att.out, att.cache.k.view(torch.uint8), att.cache.v.view(torch.uint8), out,
                                    s.committed, s.accept_len, s.out_tokens, s.out_len, s.status, att.status)]

    loop, tokens, conf, logits = make()
    calls, out, keep = whole_step(loop, tokens, conf, logits)
    out.fill_(3.0)
    eager = []
    for _ in range(2):
        for c in calls:
            c()
        eager.append(state(loop, out))
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        loop, tokens, conf, logits = make()
        calls, out, keep = whole_step(loop, tokens, conf, logits)
        out.fill_(3.0)
        graph = bd.StepGraph(stream)
        for c in calls:
            c()
        graph.end()
        for want in eager:
            graph.launch()
            stream.synchronize()
            for a, b in zip(state(loop, out), want):
                assert torch.equal(a, b)
    assert int(loop.step.status.item()) == 0 and int(loop.attention.status.item()) == 0


@gpu
def test_a_replayed_graph_takes_other_workspaces_beside_it(dev):
    """Two layers' captured calls, each with its own workspace, on two streams at once: as one after the
    other."""
    loops = [DecodeLoop(64, 4, 128, prompt=6144, max_len=64, seed=k, device=dev) for k in (1, 2)]
    want, runs = [], []
    for loop in loops:
        tokens, conf = loop.draft()
        loop.step.schedule_pack(conf, tokens)
        loop.target()
        want.append(loop.attention.out.clone())
    torch.cuda.synchronize()
    for loop in loops:
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            s = loop.step
            qkv = loop.project(loop.emb[s.packed_ids.clamp(0, loop.V - 1).long()])
            calls = loop.attention.prepare(*qkv, s.row_req, s.row_pos, s.cu, loop.lengths)
            loop.attention.out.fill_(7.0)
            graph = bd.StepGraph(stream)
            for c in calls:
                c()
            graph.end()
            runs.append((graph, stream, qkv))
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, stream, _ in runs:
            graph.launch(stream)
    torch.cuda.synchronize()
    for loop, w in zip(loops, want):
        M = int(loop.step.cu[-1])
        assert torch.equal(loop.attention.out[:M], w[:M])


@gpu
@pytest.mark.parametrize("form", ["sinks", "shared"])
@pytest.mark.parametrize("w", [3, 60])                 # units of few rows and of many
def test_pages_past_32_bit_offsets(dev, form, w):
    """The same pages in a small cache and at the end of one of more than 2^32 bytes: the same bits."""
    heads, page, dim, group = 4, 64, 128, 2
    B, prefix, own = (2, 0, 700) if form == "sinks" else (40, 6400, 90)
    rng = np.random.default_rng(w)
    front, mine = prefix // page, -(-(own + w) // page)
    n = front + B * mine
    table = np.concatenate([np.tile(np.arange(front), (B, 1)), front + np.arange(B * mine).reshape(B, mine)], 1)
    put = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(dev)      # noqa: E731
    k, v = (put(rng.integers(0, 0x78, (n, heads, page, dim), dtype=np.uint8)) for _ in range(2))
    scale = put(rng.uniform(1e-4, 1e-3, (n, heads)).astype(np.float32))
    g = torch.Generator(device=dev).manual_seed(w)
    q = torch.randn(B * w, heads * group, dim, generator=g, device=dev).bfloat16()
    i32 = dict(dtype=torch.int32, device=dev)
    cu = torch.arange(0, B * w + 1, w, **i32)
    lengths = torch.full((B,), prefix + own, **i32)
    size = bd.dspark_attend_shared_workspace_bytes(B * w, heads * group, heads, dim, B)
    ws, results = torch.empty(size, dtype=torch.uint8, device=dev), []
    for at in (0, (1 << 32) // (heads * page * dim) + 5):
        pages = [torch.zeros(at + n, heads, page, dim, dtype=torch.uint8, device=dev) for _ in range(2)]
        scales = torch.ones(at + n, heads, device=dev)
        for to, x in zip((*pages, scales), (k, v, scale)):
            to[at:] = x
        cache = bd.PagedCache(*pages, scales, scales, put((table + at).astype(np.int32)))
        out, status = torch.zeros_like(q), torch.zeros(1, **i32)
        if form == "sinks":
            bd.dspark_attend_sinks(cache, q, out, cu, lengths, ws, window=300, sinks=70, status=status)
        else:
            bd.dspark_attend_shared(cache, q, out, cu, lengths, torch.tensor([0, B], **i32),
                                    torch.tensor([prefix], **i32), ws, status=status)
        results.append(out)
        assert int(status.item()) == 0
    assert torch.isfinite(results[0]).all() and torch.equal(*results)
