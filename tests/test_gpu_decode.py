"""The operators of the target forward as a decode step runs them together: rotate in the draft,
append and attend under the packed rows of schedule_pack, lengths advanced by verify's accept
lengths; captured into a CUDA graph; on streams other than the current one."""
import numpy as np
import pytest
import torch

import cache_ref as ref
from speculative_decoding_ragged_gb300 import _binding as bd
from speculative_decoding_ragged_gb300.decode import CachedAttention, DecodeLoop

from gpu_util import device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return device()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def ints(t):
    return t.cpu().numpy().astype(np.int64)


def attention_error(att, cu, lengths, got):
    """(error, bound) of one call's output against 64 bits over what the cache holds."""
    c = att.cache
    rows = int(cu[-1])
    scales = [f64(s).reshape(c.n_pages, c.heads) for s in (c.k_scale, c.v_scale)]
    codes = [t.view(torch.uint8).cpu().numpy() for t in (c.k, c.v)]
    q = f64(att.turned)[:rows]
    want, _, spread, big, pieces = ref.attend(q, *codes, *scales, ints(c.table), lengths, cu,
                                              c.dim ** -0.5, att.window)
    # as in the operator's own test: fp32 products and sums, q's pieces, the weights' pieces, and
    # one rounding of the result
    ds = (c.dim + 8) * 2.0 ** -24 * big + 2.0 ** -17 * c.dim ** 0.5 * np.abs(q).max(-1) * 448 * scales[0].max()
    tol = spread * (np.exp(2 * ds) - 1 + 2.0 ** -20)[..., None] + pieces
    tol = tol + 2.0 ** -8 * (np.abs(want) + tol) + 1e-30
    return np.abs(f64(got)[:rows] - want), tol


@pytest.mark.parametrize("dim,page,window", [(64, 16, 0), (128, 32, 9)])
def test_loop(dev, dim, page, window):
    loop = DecodeLoop(5, 4, 512, dim=dim, page=page, window=window, seed=dim, device=dev)
    att, step = loop.attention, loop.step
    seen = set()
    for _ in range(12):
        before = ints(loop.lengths)
        tokens, conf = loop.draft()
        step.schedule_pack(conf, tokens)
        logits = loop.target()
        cu = ints(step.cu)
        err, tol = attention_error(att, cu, before, att.out)
        assert (err <= tol).all(), float((err - tol).max())
        step.verify_scatter(logits, tokens)
        L = ints(step.accept_len)
        # greedy verification over the packed rows, in words
        best = ints(logits.float().argmax(-1))
        for b in range(loop.B):
            g = best[cu[b]:cu[b + 1]]
            d = ints(tokens)[b, 1:len(g)]
            n = 1 + int(np.cumprod(g[:-1] == d).sum())
            assert L[b] == n
            assert (ints(step.committed)[b, :n] == g[:n]).all()
        loop.advance()
        assert (ints(loop.lengths) == before + L).all()
        seen.update(int(x) for x in ints(step.windows))
    assert int(step.status.item()) == 0 and int(att.status.item()) == 0
    assert (ints(step.out_len) == ints(loop.lengths)).all()
    assert len(seen) > 1                      # windows of several widths were packed


def case(dev, seed, rows=29, B=5, q_heads=8, heads=2, dim=128, page=16):
    """A layer whose requests hold 0 to 90 tokens already, and a step's packed rows."""
    rng = np.random.default_rng(seed)
    w = rng.multinomial(rows, np.ones(B) / B)
    cu = np.concatenate([[0], np.cumsum(w)]).astype(np.int32)
    lengths = rng.integers(0, 90, B).astype(np.int32)
    blocks = 10
    put = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(dev)
    table = put(rng.permutation(B * blocks).astype(np.int32).reshape(B, blocks))
    att = CachedAttention(max(rows, int(lengths.sum())), q_heads, heads, dim, table, B * blocks, page,
                          bd.Rope.make(dim, device=dev))
    def packed(n):
        req = np.repeat(np.arange(B), n).astype(np.int32)
        pos = np.concatenate([np.arange(x) for x in n]).astype(np.int32)
        t = lambda h: put(rng.standard_normal((int(n.sum()), h, dim)).astype(np.float32)).bfloat16()
        return [t(q_heads), t(heads), t(heads), put(req), put(pos),
                put(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))]
    att.run(*packed(lengths), torch.zeros(B, dtype=torch.int32, device=dev))       # the prompts
    return att, packed(w), put(lengths)


def state(att):
    return [t.clone() for t in (att.out, att.turned, att.cache.k.view(torch.uint8),
                                att.cache.v.view(torch.uint8), att.cache.k_scale, att.cache.v_scale,
                                att.status)]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_repeats_bit_for_bit(dev):
    att, rows, lengths = case(dev, 1)
    att.run(*rows, lengths)
    first = state(att)
    err, tol = attention_error(att, ints(rows[5]), ints(lengths), att.out)
    assert (err <= tol).all()
    att.run(*rows, lengths)
    assert same(first, state(att))


@pytest.mark.parametrize("size", [dict(), dict(rows=400, page=64)])      # windows; prompts
def test_graph_replays_eager_steps(dev, size):
    att, rows, lengths = case(dev, 2, **size)
    side = torch.cuda.Stream(device=dev)
    other, orows, olen = case(dev, 2, **size)  # the same case, run eagerly
    assert same(state(att), state(other))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        calls = att.prepare(*rows, lengths)
        graph = bd.StepGraph(side)
        try:
            for call in calls:
                call()
        finally:
            graph.end()
    replay = graph.prepare_launch()
    for step in range(4):
        # new inputs into the same tensors: other lengths, another split of the rows
        att2, fresh, flen = case(dev, 10 + step, **size)
        for dst, odst, src in zip([*rows, lengths], [*orows, olen], [*fresh, flen]):
            dst.copy_(src)
            odst.copy_(src)
        for a in (att, other):
            for name in ("k", "v", "k_scale", "v_scale", "table"):
                getattr(a.cache, name).view(torch.uint8).copy_(getattr(att2.cache, name).view(torch.uint8))
        torch.cuda.synchronize()
        replay()
        other.run(*orows, olen)
        torch.cuda.synchronize()
        assert same(state(att), state(other)), step
        err, tol = attention_error(att, ints(rows[5]), ints(lengths), att.out)
        assert (err <= tol).all()


@pytest.mark.parametrize("size", [dict(), dict(rows=400, page=64)])
def test_another_stream(dev, size):
    """Calls follow the stream they are given, not the stream their tensors came from."""
    att, rows, lengths = case(dev, 3, **size)
    want, wrows, wlen = case(dev, 3, **size)
    want.run(*wrows, wlen)
    late = rows[0].clone()
    rows[0].zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream(device=dev)
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)          # a millisecond: work of the default stream would pass
        rows[0].copy_(late)
        att.run(*rows, lengths)
    side.synchronize()
    assert same(state(att), state(want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rotate_gradient_by_differences(dev, dtype):
    """inverse is the gradient: <rotate(x + h d) - rotate(x - h d), w> / 2h = <d, inverse(w)>.
    Rotation is linear, so the difference is exact but for the roundings counted below."""
    gen = torch.Generator().manual_seed(5)
    rows, heads, dim = 7, 3, 64
    rope = bd.Rope.make(dim, scaling="linear", factor=2.0, mscale=1.25, device=dev)
    pos = torch.tensor([0, 1, 77, 4095, 131071, 2 ** 31 - 1, -5], dtype=torch.int32, device=dev)
    x, d, w = (torch.randn(rows, heads, dim, generator=gen).to(dev, dtype) for _ in range(3))

    def turn(t, inverse=False):
        y = torch.empty_like(t)
        bd.dspark_rotate(t, y, pos, rope, inverse=inverse)
        return y.double()
    plus, minus = (x + d).to(dtype), (x - d).to(dtype)
    step = (plus.double() - minus.double()) / 2          # the step that was taken, exactly
    lhs = ((turn(plus) - turn(minus)) / 2 * w.double()).sum((1, 2))
    rhs = (step * turn(w, inverse=True)).sum((1, 2))
    # per element: half a step of the type, and the rotation's own error (cache_ref.ROTATE_TOL)
    eps = torch.finfo(dtype).eps / 2 + 2 * ref.ROTATE_TOL
    size = 1.25 * 2 ** 0.5
    bound = eps * size * (((plus.abs() + minus.abs()).double().amax((1, 2)) * w.double().abs().sum((1, 2))) +
                          step.abs().sum((1, 2)) * w.double().abs().amax((1, 2)) * 1.0)
    assert ((lhs - rhs).abs() <= bound).all(), (lhs - rhs, bound)


@pytest.mark.parametrize("rows,dim,dtype", [(29, 128, torch.bfloat16), (400, 128, torch.bfloat16),
                                            (29, 128, torch.float32)])
def test_cache_past_32_bits(dev, rows, dim, dtype):
    """Pages whose codes lie more than 2^32 bytes into the cache: the same bits as in a small one."""
    small, packed, lengths = case(dev, 4, rows=rows, dim=dim, page=64)
    heads, page = 2, 64
    per = heads * page * dim
    pages = small.cache.n_pages
    n = (2 ** 32 + per - 1) // per + pages + 1
    assert (n - pages) * per > 2 ** 32
    big = CachedAttention(small.out.shape[0], small.out.shape[1], heads, dim,
                          small.cache.table + (n - pages), 1, page, small.rope, dtype=dtype)
    k, v = (torch.empty(n, heads, page, dim, dtype=torch.uint8, device=dev) for _ in range(2))
    ks, vs = (torch.ones(n, heads, device=dev) for _ in range(2))
    other = CachedAttention(small.out.shape[0], small.out.shape[1], heads, dim, small.cache.table,
                            pages, page, small.rope, dtype=dtype)
    for name, t in (("k", k), ("v", v), ("k_scale", ks), ("v_scale", vs)):
        src = getattr(small.cache, name)
        t[n - pages:].view(torch.uint8).copy_(src.view(torch.uint8))
        getattr(other.cache, name).view(torch.uint8).copy_(src.view(torch.uint8))
    big.cache = bd.PagedCache(k, v, ks, vs, big.cache.table)
    args = [t.to(dtype) for t in packed[:3]] + packed[3:] + [lengths]
    a, b = other.run(*args), big.run(*args)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and bool(a.float().abs().sum() > 0)
    assert torch.equal(other.cache.k.view(torch.uint8), k[n - pages:])
    assert torch.equal(other.cache.v.view(torch.uint8), v[n - pages:])
    assert int(big.status.item()) == 0
