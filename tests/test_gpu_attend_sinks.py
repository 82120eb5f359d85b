"""dspark_attend_sinks against 64 bits: windows and sinks of every size against each other and the
contexts, both kinds of tensor-core kernel, fp32 and other head sizes; entries of the pages between
that are stale, pages out of range, queries that are no numbers, strides, graphs; the same bits as
dspark_attend where nothing is left out; the refusals."""
import ctypes

import numpy as np
import pytest
import torch

import forms_ref
from speculative_decoding_ragged_gb300 import _binding as bd
from test_gpu_attend import BOTH, Case

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_ragged_gb300 import build
    build.build()
    return bd.lib()


def test_refuses_on_the_host(lib):
    P = ctypes.c_void_p
    c = bd._Cache(4096, 4096, 4096, 4096, 4096, 8, 2, 16, 64, 4)

    def call(q=4096, hq=4, dt=0, rows=3, B=2, scale=0.1, window=5, sinks=1, ws=4096, wb=1 << 30):
        rc = lib.dspark_attend_sinks(ctypes.byref(c), P(q), 256, P(4096), 256, hq, dt, rows, P(4096), P(4096), B,
                                     scale, window, sinks, P(None), P(ws), wb, None, None)
        return rc, bd.last_error()

    for code, kw, word in [(-1, dict(sinks=-1), "sinks"), (-1, dict(sinks=2 ** 31 - 1), "sinks"),
                           (-1, dict(window=-1), "window=-1"), (-1, dict(hq=3), "q_heads"),
                           (-1, dict(dt=9), "dtype"), (-1, dict(q=None), "required"),
                           (-1, dict(scale=float("nan")), "scale"), (-1, dict(wb=1), "workspace"),
                           (-1, dict(ws=4104), "workspace"), (-1, dict(rows=-1), "rows=-1")]:
        rc, msg = call(**kw)
        assert rc == code and msg.startswith("dspark_attend_sinks") and word in msg, (kw, rc, msg)
    assert call(rows=0, q=None)[0] == 0 and call(B=0)[0] == 0


class Sinks(Case):
    def go(self, dtype, window, sinks, *, plain=False, strides=False, prepare=False, lse=True):
        dev = torch.device("cuda:0")
        t = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(dev)     # noqa: E731
        cache = bd.PagedCache(t(self.codes["k"]), t(self.codes["v"]), t(self.scale["k"]), t(self.scale["v"]),
                              t(self.table))
        q = torch.as_tensor(self.q).to(dtype).to(dev)
        if strides:
            q = torch.cat([q, torch.full_like(q, float("nan"))], 1)[:, :self.hq]
        out = torch.full((self.rows, self.hq + (2 if strides else 0), self.dim), 5.0, dtype=dtype, device=dev)
        out = out[:, :self.hq]
        ls = torch.full((self.rows, self.hq), 5.0, device=dev) if lse else None
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        ws = torch.full((bd.dspark_attend_workspace_bytes(self.heads, self.dim),), 0xAA, dtype=torch.uint8, device=dev)
        cu, lengths = t(self.cu), t(self.lengths)
        if plain:
            bd.dspark_attend(cache, q, out, cu, lengths, ws, window=window, lse=ls, status=st)
        else:
            call = bd.dspark_attend_sinks(cache, q, out, cu, lengths, ws, window=window, sinks=sinks, lse=ls,
                                          status=st, prepare=True)
            if prepare:
                return call, q, out, ls, (cache, ws, cu, lengths, st)
            call()
            call()                           # the second call finds the first's workspace
        torch.cuda.synchronize()
        return q.double().cpu().numpy(), out.double().cpu().numpy(), \
            ls.double().cpu().numpy() if lse else None, int(st.item())

    def seen(self, window, sinks):
        def tokens(b, pos):
            t = np.arange(pos + 1)
            return t[(t > pos - window) | (t < sinks)] if window else t
        return tokens

    def hold(self, dtype, window, sinks, status=0, **kw):
        q, out, lse, st = self.go(dtype, window, sinks, **kw)
        assert st == status
        forms_ref.check(self, dtype, q, out, lse, self.seen(window, sinks))
        return out, lse


# w, lengths, heads, group, dim, page: single tokens, windows of one and several units, prompts (the
# wide kernel), contexts of nothing to many tiles
SHAPES = [([1], [0], 1, 1, 64, 16), ([1] * 6, [0, 1, 127, 128, 700, 1500], 2, 8, 128, 32),
          ([4, 0, 7, 2], [5, 300, 1000, 129], 2, 3, 64, 16), ([5], [5000], 1, 6, 128, 64),
          ([16, 3], [2500, 40], 2, 4, 128, 128), ([150, 1, 40], [600, 900, 0], 1, 4, 64, 32),
          ([300], [1], 1, 1, 128, 16), ([70, 33], [1, 1500], 2, 2, 128, 64)]


@gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 1), (16, 4), (100, 19), (129, 128), (300, 300), (40, 1000), (2000, 5)])
def test_sinks(lib, shape, window, sinks):
    Sinks(sum(shape[0]) + window, *shape).hold(torch.bfloat16, window, sinks)


@gpu
@pytest.mark.parametrize("shape,window,sinks", [(SHAPES[1], 16, 4), (SHAPES[2], 100, 40), (SHAPES[4], 33, 32),
                                                (SHAPES[2], 1, 700), (([3, 9], [200, 31], 2, 5, 48, 16), 20, 3),
                                                (([2, 1], [90, 400], 1, 4, 256, 16), 64, 33)])
@pytest.mark.parametrize("dtype", BOTH)
def test_any_size(lib, shape, window, sinks, dtype):
    if dtype == torch.bfloat16 and shape[4] in (64, 128):
        dtype = torch.float32
    Sinks(7, *shape).hold(dtype, window, sinks)


@gpu
@pytest.mark.parametrize("dtype", BOTH)
def test_pages_between_are_not_looked_at(lib, dtype):
    c = Sinks(3, [1, 5, 30, 150], [0, 1000, 131, 700], 2, 3, 64, 16)
    window, sinks = 100, 21
    for b in range(4):
        gone = (int(c.lengths[b]) - window + 1) // 16
        if gone > 2:
            c.table[b, 2:gone] = -1
    c.hold(dtype, window, sinks)


@gpu
@pytest.mark.parametrize("dtype", BOTH)
def test_bad_pages(lib, dtype):
    c = Sinks(4, [2, 3, 40], [400, 200, 300], 2, 2, 128, 16)
    c.table[0, 0] = c.n                       # the sinks' page
    c.table[1, 12] = -1                       # one of the window's
    c.table[2, 0] = 10 ** 6
    c.hold(dtype, 37, 16, status=bd.STATUS_BAD_PAGE)
    c = Sinks(5, [1], [200], 1, 4, 128, 16)
    c.table[0] = -1                           # nothing there at all
    _, lse = c.hold(dtype, 10, 3, status=bd.STATUS_BAD_PAGE)
    assert np.isneginf(lse[0]).all()


@gpu
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[5]])
@pytest.mark.parametrize("dtype", BOTH)
def test_the_same_bits_as_attend(lib, shape, dtype):
    """Without a window, without sinks."""
    c = Sinks(6, *shape)
    for window, sinks in ((0, 7), (50, 0)):
        a, b = c.go(dtype, window, sinks), c.go(dtype, window, 0, plain=True)
        np.testing.assert_array_equal(a[1], b[1])
        np.testing.assert_array_equal(a[2], b[2])


@gpu
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[5]])
def test_queries_that_are_no_numbers(lib, shape):
    c = Sinks(8, *shape)
    _, clean, _, _ = c.go(torch.bfloat16, 60, 9)
    c.q[2, 1, 5], c.q[4, 2, 0] = np.nan, np.inf
    _, out, _, _ = c.go(torch.bfloat16, 60, 9)
    hit = np.zeros(out.shape[:2], bool)
    hit[2, 1] = hit[4, 2] = True
    assert np.isnan(out[hit]).all()
    np.testing.assert_array_equal(out[~hit], clean[~hit])


@gpu
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[5]])
@pytest.mark.parametrize("dtype", BOTH)
def test_strides_and_no_lse(lib, shape, dtype):
    c = Sinks(9, *shape)
    out, _ = c.hold(dtype, 64, 8)
    np.testing.assert_array_equal(c.go(dtype, 64, 8, strides=True)[1], out)
    np.testing.assert_array_equal(c.go(dtype, 64, 8, lse=False)[1], out)


@gpu
@pytest.mark.parametrize("shape", [SHAPES[1], SHAPES[7]])
def test_graph_on_another_stream(lib, shape):
    c = Sinks(10, *shape)
    want = c.go(torch.bfloat16, 200, 6)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call, q, out, lse, keep = c.go(torch.bfloat16, 200, 6, prepare=True)
        graph = bd.StepGraph(stream)
        call()
        graph.end()
    stream.synchronize()
    assert (out == 5).all()
    for _ in range(2):
        graph.launch()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(out.double().cpu().numpy(), want[1])
    np.testing.assert_array_equal(lse.double().cpu().numpy(), want[2])


@gpu
@pytest.mark.parametrize("seed", range(10))
def test_random_shapes(lib, seed):
    rng = np.random.default_rng(300 + seed)
    B = int(rng.integers(1, 8))
    w = rng.integers(0, 9, B) if seed % 3 else rng.integers(0, 120, B)
    w[0] = max(w[0], 1)
    c = Sinks(seed, w, rng.integers(0, 1200, B), int(rng.integers(1, 4)), int(rng.integers(1, 9)),
              int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 128])), spread=2.0)
    c.hold(torch.bfloat16, int(rng.integers(1, 500)), int(rng.integers(1, 400)))
