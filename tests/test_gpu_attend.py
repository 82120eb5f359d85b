"""dspark_attend against 64-bit attention over the same codes and scales: bf16 and fp32, shared
heads, every page size, windows and lengths from none to many, sliding windows, several row tiles
and splits; stale slots full of NaN, pages out of range, rows that see nothing, strided rows,
streams and graphs; the refusals. Tolerances count the roundings that the header names."""
import ctypes

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


def test_attend_refuses_on_the_host(lib):
    P = ctypes.c_void_p

    def cache(n=8, heads=2, page=16, dim=64, width=4, k=4096):
        return bd._Cache(k, 4096, 4096, 4096, 4096, n, heads, page, dim, width)

    def call(c=cache(), q=4096, qs=256, out=4096, os=256, hq=4, dt=0, rows=3, cu=4096,
             lengths=4096, B=2, scale=0.1, window=0, lse=None, ws=4096, wb=1 << 30):
        rc = lib.dspark_attend(ctypes.byref(c) if c is not None else None, P(q), qs, P(out), os, hq,
                               dt, rows, P(cu), P(lengths), B, scale, window, P(lse), P(ws), wb,
                               None, None)
        return rc, bd.last_error()

    for code, kw, word in [
            (-1, dict(c=None), "cache"), (-2, dict(c=cache(page=8)), "page"),
            (-2, dict(c=cache(dim=24)), "dim"), (-1, dict(c=cache(k=None)), "pages"),
            (-1, dict(dt=9), "dtype"), (-1, dict(rows=-1), "rows=-1"), (-1, dict(B=-2), "B=-2"),
            (-1, dict(window=-1), "window=-1"), (-1, dict(hq=3), "q_heads"),
            (-1, dict(hq=0), "q_heads"), (-2, dict(rows=2 ** 29), "too large"),
            (-1, dict(qs=255), "row strides"), (-1, dict(os=255), "row strides"),
            (-1, dict(scale=float("inf")), "scale"), (-1, dict(scale=float("nan")), "scale"),
            (-1, dict(q=None), "required"), (-1, dict(out=None), "required"),
            (-1, dict(cu=None), "required"), (-1, dict(lengths=None), "required"),
            (-1, dict(q=4097), "required"), (-1, dict(lse=4098), "required"),
            (-1, dict(ws=None), "workspace"), (-1, dict(ws=4104), "workspace"),
            (-1, dict(wb=1), "workspace")]:
        rc, msg = call(**kw)
        assert rc == code and msg.startswith("dspark_attend") and word in msg, (kw, rc, msg)
    assert call(rows=0, q=None, out=None)[0] == 0 and call(B=0, cu=None)[0] == 0
    assert bd.dspark_attend_workspace_bytes(8, 128) <= 64 << 20
    for bad in ((0, 64), (1, 0), (1, 24), (1, 512)):
        assert bd.dspark_attend_workspace_bytes(*bad) == 0 and "bad sizes" in bd.last_error()


class Case:
    def __init__(self, seed, w, lengths, heads, group, dim, page, spread=1.0, sharp=1.0, pad=2):
        rng = np.random.default_rng(seed)
        self.w, self.lengths = np.asarray(w), np.asarray(lengths, np.int32)
        self.heads, self.hq, self.dim, self.page = heads, heads * group, dim, page
        B = len(w)
        blocks = [-(-(int(n) + int(c)) // page) for n, c in zip(w, lengths)]
        self.n = sum(blocks) + 2
        order = rng.permutation(self.n)
        self.table = np.full((B, max(max(blocks), 1)), -7, np.int32)
        x = {s: rng.standard_normal((self.n, heads, page, dim)) *
             np.exp2(rng.uniform(-spread, spread, (self.n, heads, 1, 1))) for s in "kv"}
        self.codes, self.scale = {}, {}
        for s in "kv":
            sc = np.exp2(np.ceil(np.log2(np.abs(x[s]).max(axis=(2, 3)) / 448.0)))
            self.scale[s] = sc.astype(np.float32)
            self.codes[s] = ref.encode(x[s] / sc[:, :, None, None])
        k = 0
        for b, m in enumerate(blocks):
            self.table[b, :m] = order[k:k + m]
            k += m
            if m:                            # slots past the last token: NaN codes
                used = int(lengths[b]) + int(w[b]) - (m - 1) * page
                for s in "kv":
                    self.codes[s][order[k - 1], :, used:] = 0x7f if s == "k" else 0xff
        self.cu = np.concatenate([[0], np.cumsum(w)]).astype(np.int32)
        self.rows = int(self.cu[-1]) + pad
        self.q = rng.standard_normal((self.rows, self.hq, dim)) * sharp

    def run(self, dtype, window=0, scale=None, strides=False, lse=True, ws_fill=0xAA, prepare=None):
        dev = torch.device("cuda:0")
        t = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(dev)     # noqa: E731
        cache = bd.PagedCache(t(self.codes["k"]), t(self.codes["v"]), t(self.scale["k"]),
                              t(self.scale["v"]), t(self.table))
        q = torch.as_tensor(self.q).to(dtype).to(dev)
        if strides:                          # rows of a wider buffer, on both sides
            q = torch.cat([q, torch.full_like(q, float("nan"))], 1)[:, :self.hq]
        out = torch.full((self.rows, self.hq + (2 if strides else 0), self.dim), 5.0, dtype=dtype,
                         device=dev)[:, :self.hq]
        ls = torch.full((self.rows, self.hq), 5.0, device=dev) if lse else None
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        nb = bd.dspark_attend_workspace_bytes(self.heads, self.dim)
        ws = torch.full((nb,), ws_fill, dtype=torch.uint8, device=dev)
        for _ in range(2):                   # twice: the second call finds the first's workspace
            bd.dspark_attend(cache, q, out, t(self.cu), t(self.lengths), ws, scale=scale,
                             window=window, lse=ls, status=st)
        torch.cuda.synchronize()
        qh = q.double().cpu().numpy()
        return (qh, out.double().cpu().numpy(), ls.double().cpu().numpy() if lse else None,
                int(st.item()))

    def check(self, dtype, window=0, scale=None, status=0, **kw):
        q, out, lse, st = self.run(dtype, window, scale, **kw)
        a = self.dim ** -0.5 if scale is None else scale
        want, wl, spread, big, pieces = ref.attend(q, self.codes["k"], self.codes["v"], self.scale["k"],
                                           self.scale["v"], self.table, self.lengths, self.cu, a,
                                           window)
        M = int(self.cu[-1])
        assert st == status
        assert (out[M:] == 5.0).all()
        # a score: dim products and sums in fp32 (each within 2^-24 of scale * sum |q k|; the
        # factors' roundings a few more), and on the tensor cores q's pieces, 2^-17 of the row's
        # largest element, at most 2^-17 dim of scale * max|q| max|k|
        fast = dtype == torch.bfloat16 and self.dim in (64, 128)
        ds = (self.dim + 8) * 2.0 ** -24 * big
        if fast:
            kmax = (448.0 * self.scale["k"]).max()
            ds = ds + 2.0 ** -17 * self.dim * abs(a) * np.abs(q).max(-1) * kmax
        ds = ds[:M]
        # exp2, the sums' order and the division: 2^-20 together
        rel = (np.exp(2 * ds) - 1 + 2.0 ** -20)[..., None]
        tol = spread[:M] * rel
        if fast:
            tol = tol + pieces[:M]
        tol = tol + torch.finfo(dtype).eps / 2 * (np.abs(want[:M]) + tol) + 1e-30
        err = np.abs(out[:M] - want[:M])
        assert (err <= tol).all(), (float(err.max()), float((err - tol).max()))
        empty = np.isneginf(wl[:M])
        assert (out[:M][empty] == 0).all()
        if lse is not None:
            assert (np.isneginf(lse[:M]) == empty).all()
            e = np.abs(np.where(empty, 0, lse[:M]) - np.where(empty, 0, wl[:M]))
            assert (e <= 2 * ds + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, wl[:M])))).all(), e.max()
            assert (lse[M:] == 5.0).all()
        return out, lse


BOTH = [torch.bfloat16, torch.float32]
CASES = [
    # w, lengths, heads, group, dim, page
    ([1], [0], 1, 1, 64, 16),
    ([1], [0], 1, 1, 128, 128),
    ([4], [1000], 2, 4, 128, 16),
    ([1, 8, 3, 5, 2], [0, 15, 16, 127, 128], 2, 3, 64, 16),
    ([3, 1, 7], [129, 255, 640], 3, 1, 128, 32),
    ([0, 2, 0, 1], [7, 300, 0, 126], 2, 8, 64, 64),
    ([40], [100], 1, 4, 128, 64),            # 160 rows of one head: two tiles of 128
    ([33, 70], [1, 500], 2, 2, 64, 128),
    ([200], [0], 1, 1, 128, 16),
    ([1] * 50, [3 * i for i in range(50)], 2, 2, 128, 16),
    ([5], [5000], 1, 7, 64, 16),             # split over many CTAs and joined
    ([16, 1], [2500, 1], 8, 4, 128, 32),
    ([9], [77], 2, 16, 128, 64),             # 144 rows: a tile ends inside a position's heads
]


@gpu
@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("case", CASES)
def test_attend(lib, case, dtype):
    Case(sum(case[0]) + case[4], *case).check(dtype)


PROMPTS = [
    # w, lengths, heads, group, dim, page, window: requests of many units of 128 rows, and the
    # threads that count them from 32 for one request down to one for two requests
    ([1100, 0, 5], [3, 9, 200], 1, 4, 64, 16, 0),
    ([1100], [0], 1, 4, 128, 64, 100),
    ([40, 61, 300, 1, 0, 90, 33], [0, 127, 5, 600, 7, 64, 1], 2, 3, 64, 32, 0),
    ([13] * 60, [7 * i for i in range(60)], 1, 4, 64, 16, 0),
    ([12] * 200, [i % 90 for i in range(200)], 1, 4, 64, 16, 0),
    ([129, 257], [1000, 3], 3, 1, 128, 32, 40),
    ([90], [2900], 1, 16, 128, 128, 0),
]


@gpu
@pytest.mark.parametrize("case", PROMPTS)
def test_prompts(lib, case):
    c = Case(sum(case[0]) + case[6], *case[:6])
    c.check(torch.bfloat16, case[6])
    c.q *= 5.0                               # one token takes nearly all: maxima rise from tile to tile
    c.check(torch.bfloat16, case[6])


@gpu
def test_prompts_with_bad_pages_and_queries(lib):
    c = Case(21, [70, 50], [300, 0], 2, 4, 128, 16)
    c.table[0, 3] = -1
    c.table[1, 0] = c.n                      # request 1's first rows see nothing
    out, lse = c.check(torch.bfloat16, status=bd.STATUS_BAD_PAGE)
    assert np.isneginf(lse[c.cu[1]:c.cu[1] + 16]).all()
    q = c.q.copy()
    c.q[33, 5, 7], c.q[100, 0, 0] = np.nan, -np.inf
    _, bad, _, _ = c.run(torch.bfloat16)
    c.q = q
    hit = np.zeros(out.shape[:2], bool)
    hit[33, 5] = hit[100, 0] = True
    assert np.isnan(bad[hit]).all()
    np.testing.assert_array_equal(bad[~hit], out[~hit])


@gpu
@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("window", [1, 2, 16, 100, 129, 1000])
def test_sliding_window(lib, window, dtype):
    c = Case(window, [1, 5, 30, 150], [0, 1000, 131, 300], 2, 3, 64, 16)
    # entries of pages before every row's window may be stale: they are not looked at
    for b in range(4):
        gone = (int(c.lengths[b]) - window + 1) // 16
        if gone > 0:
            c.table[b, :gone] = -1
    c.check(dtype, window)


@gpu
@pytest.mark.parametrize("dtype", BOTH)
def test_sharp_and_flat_scores(lib, dtype):
    """One token that takes nearly all the weight, wherever it sits; equal scores; large scales."""
    c = Case(3, [3, 6], [700, 129], 2, 4, 128, 32, sharp=6.0)
    c.check(dtype)
    c.check(dtype, scale=-0.3)
    c.check(dtype, scale=0.0)
    c.q[:] = 0.0
    c.check(dtype)


@gpu
@pytest.mark.parametrize("dtype", BOTH)
def test_blocks_of_very_different_scales(lib, dtype):
    """Values of one block 2^40 larger than another's, and scales that are no powers of two."""
    c = Case(5, [4, 2], [400, 90], 2, 2, 64, 16)
    rng = np.random.default_rng(0)
    c.scale["v"] *= np.exp2(rng.integers(-20, 20, c.scale["v"].shape)).astype(np.float32)
    c.check(dtype)
    c.scale["k"] *= rng.uniform(0.5, 1.5, c.scale["k"].shape).astype(np.float32)
    c.scale["v"] *= rng.uniform(0.5, 1.5, c.scale["v"].shape).astype(np.float32)
    c.check(dtype)


@gpu
@pytest.mark.parametrize("dtype", BOTH)
def test_pages_out_of_range_are_not_seen(lib, dtype):
    c = Case(6, [2, 3, 2], [100, 200, 3], 2, 2, 128, 16)
    c.table[0, 1] = c.n                       # in the middle
    c.table[1, 12] = -1                       # the last full one
    c.table[2, 0] = 10 ** 6                   # all there is: these rows see nothing
    out, lse = c.check(dtype, status=bd.STATUS_BAD_PAGE)
    assert np.isneginf(lse[c.cu[2]:c.cu[3]]).all()
    # a request longer than the table is wide
    c = Case(6, [2], [100], 2, 2, 128, 16)
    c.table = np.ascontiguousarray(c.table[:, :4])
    c.check(dtype, status=bd.STATUS_BAD_PAGE)


@gpu
@pytest.mark.parametrize("dtype", BOTH)
def test_rows_and_lengths_out_of_range(lib, dtype):
    c = Case(7, [2, 2], [0, 50], 2, 2, 64, 16)
    want_q, want, _, _ = c.run(dtype)
    c.lengths[0] = -3                         # counts as 0
    _, out, _, st = c.run(dtype)
    assert st == bd.STATUS_BAD_LENGTH
    np.testing.assert_array_equal(out, want)
    c.lengths[0] = 0
    c.cu[2] = c.rows + 5                      # request 1's rows leave the buffer
    _, out, _, st = c.run(dtype)
    assert st == bd.STATUS_BAD_ROWS
    np.testing.assert_array_equal(out[:2], want[:2])
    assert (out[2:] == 5.0).all()


@gpu
@pytest.mark.parametrize("dtype", BOTH)
def test_strided_rows_and_no_lse(lib, dtype):
    c = Case(8, [3, 6], [50, 300], 2, 3, 128, 16)
    out, _ = c.check(dtype)
    for kw in (dict(strides=True), dict(lse=False), dict(ws_fill=0xFF)):
        again, _ = c.check(dtype, **kw)
        np.testing.assert_array_equal(again, out)     # the same bits, whatever is around


@gpu
def test_nan_and_infinite_queries_stay_in_their_row(lib):
    c = Case(9, [6], [300], 1, 4, 128, 16)
    for dtype in BOTH:
        _, clean, _, _ = c.run(dtype)
        q = c.q.copy()
        c.q[2, 1, 5] = np.nan
        c.q[4, 3, 0] = np.inf
        _, out, _, _ = c.run(dtype)
        c.q = q
        bad = np.zeros(out.shape[:2], bool)
        bad[2, 1] = bad[4, 3] = True
        assert np.isnan(out[bad]).all()
        np.testing.assert_array_equal(out[~bad], clean[~bad])


@gpu
@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(lib, seed):
    rng = np.random.default_rng(100 + seed)
    B = int(rng.integers(1, 9))
    w = rng.integers(0, 9, B) if seed % 3 else rng.integers(0, 120, B)
    lengths = rng.integers(0, 900, B)
    heads, group = int(rng.integers(1, 4)), int(rng.integers(1, 9))
    if w.sum() == 0:
        w[0] = 1
    c = Case(seed, w, lengths, heads, group, int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 128])),
             spread=2.0)
    c.check(torch.bfloat16, window=int(rng.choice([0, 0, 37, 400])))


@gpu
@pytest.mark.parametrize("dim", [16, 48, 96, 192, 256])
def test_other_head_sizes(lib, dim):
    for dtype in BOTH:
        Case(dim, [3, 1], [40, 200], 2, 5, dim, 16).check(dtype)
