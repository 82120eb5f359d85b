"""dspark_append against the 64-bit definition: without a rotation bit for bit (codes, scales,
untouched slots), with one within the rotation's rounding; both types, every page size, windows
that start, end and cross pages, empty requests, padding rows, retained codes under a growing
scale, non-finite elements, pages and rows out of range; queries on the way; the refusals."""
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


def test_append_refuses_on_the_host(lib):
    P = ctypes.c_void_p

    def cache(k=4096, v=4096, ks=4096, vs=4096, table=4096, n=8, heads=2, page=16, dim=64, width=4):
        return bd._Cache(k, v, ks, vs, table, n, heads, page, dim, width)

    def call(c=cache(), rope=None, k=4096, ks=128, v=4096, vs=128, q=4096, qs=256, qo=4096,
             os=256, hq=4, dt=0, rows=3, req=4096, pos=4096, lengths=4096, B=2):
        rc = lib.dspark_append(ctypes.byref(c) if c is not None else None,
                               ctypes.byref(rope) if rope is not None else None, P(k), ks, P(v), vs,
                               P(q), qs, P(qo), os, hq, dt, rows, P(req), P(pos), P(lengths), B,
                               None, None)
        return rc, bd.last_error()

    for code, kw, word in [
            (-1, dict(c=None), "cache"), (-1, dict(c=cache(n=-1)), "n_pages=-1"),
            (-1, dict(c=cache(heads=0)), "heads=0"), (-1, dict(c=cache(width=-1)), "width=-1"),
            (-2, dict(c=cache(page=48)), "page = 48"), (-2, dict(c=cache(page=256)), "page = 256"),
            (-2, dict(c=cache(dim=72)), "dim = 72"), (-2, dict(c=cache(dim=272)), "dim = 272"),
            (-2, dict(c=cache(heads=65536)), "heads = 65536"),
            (-2, dict(c=cache(n=2 ** 30)), "overflows"), (-1, dict(c=cache(k=None)), "pages and"),
            (-1, dict(c=cache(vs=None)), "pages and"), (-1, dict(c=cache(table=None)), "table"),
            (-1, dict(c=cache(v=4104)), "aligned"), (-1, dict(rope=bd._Rope(4096, 66, 0, 1.0)), "rot"),
            (-1, dict(dt=2), "dtype"), (-1, dict(rows=-1), "rows=-1"), (-1, dict(B=-1), "B=-1"),
            (-1, dict(ks=127), "row strides"), (-1, dict(vs=127), "row strides"),
            (-1, dict(q=None), "both"), (-1, dict(qo=None), "both"), (-1, dict(hq=0), "q_heads"),
            (-1, dict(qs=255), "q_heads"), (-1, dict(os=255), "q_heads"),
            (-2, dict(rows=2 ** 29), "too large"), (-1, dict(k=None), "required"),
            (-1, dict(v=None), "required"), (-1, dict(req=None), "required"),
            (-1, dict(pos=None), "required"), (-1, dict(lengths=None), "required"),
            (-1, dict(k=4097), "required")]:
        rc, msg = call(**kw)
        assert rc == code and msg.startswith("dspark_append") and word in msg, (kw, rc, msg)
    assert call(rows=0, k=None, v=None, req=None, pos=None)[0] == 0


class Case:
    """B requests with windows w and lengths len over shuffled pages; k, v, q rows of one
    projection; a cache as earlier steps left it."""

    def __init__(self, seed, w, lengths, heads, group, dim, page, dtype, pad=3, spread=3.0):
        rng = np.random.default_rng(seed)
        self.w, self.lengths = np.asarray(w), np.asarray(lengths, np.int32)
        self.heads, self.group, self.dim, self.page = heads, group, dim, page
        B = len(w)
        blocks = [-(-(int(n) + int(c)) // page) + 1 for n, c in zip(w, lengths)]
        self.n = sum(blocks) + 2
        order = rng.permutation(self.n)
        self.table = np.zeros((B, max(blocks)), np.int32)
        k = 0
        for b, m in enumerate(blocks):
            self.table[b, :m] = order[k:k + m]
            k += m
        req = np.repeat(np.arange(B), w)
        pos = np.concatenate([np.arange(x) for x in w] + [np.zeros(0, int)])
        self.req = np.concatenate([req, -np.ones(pad)]).astype(np.int32)
        self.pos = np.concatenate([pos, -np.ones(pad)]).astype(np.int32)
        self.rows = len(self.req)
        self.dtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        cols = heads * (group + 2)
        proj = rng.standard_normal((self.rows, cols, dim)) * \
            np.exp2(rng.uniform(-spread, spread, (self.rows, cols, 1)))
        self.proj = torch.as_tensor(proj).to(self.dtype)
        self.codes = {x: rng.integers(0, 256, (self.n, heads, page, dim)).astype(np.uint8)
                      for x in "kv"}
        for c in self.codes.values():
            c[(c & 0x7f) == 0x7f] = 0x11          # a token that counts holds no NaN
        self.scale = {x: np.exp2(rng.integers(-9, -1, (self.n, heads))).astype(np.float32)
                      for x in "kv"}

    def run(self, rope, with_q=True, times=1):
        dev = torch.device("cuda:0")
        t = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(dev)     # noqa: E731
        cache = bd.PagedCache(t(self.codes["k"]), t(self.codes["v"]), t(self.scale["k"]),
                              t(self.scale["v"]), t(self.table))
        proj = self.proj.to(dev)
        hq = self.heads * self.group
        q, k, v = proj[:, :hq], proj[:, hq:hq + self.heads], proj[:, hq + self.heads:]
        q_out = torch.full((self.rows, hq, self.dim), 9.0, dtype=self.dtype, device=dev)
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        for _ in range(times):
            bd.dspark_append(cache, k, v, t(self.req), t(self.pos), t(self.lengths), rope=rope,
                             q=q if with_q else None, q_out=q_out if with_q else None, status=st)
        torch.cuda.synchronize()
        return dict(k=cache.k.cpu().numpy(), v=cache.v.cpu().numpy(), ks=cache.k_scale.cpu().numpy(),
                    vs=cache.v_scale.cpu().numpy(), q=q_out.double().cpu().numpy(),
                    status=int(st.item()))

    def want(self, turns=None, mscale=1.0, inter=False):
        hq = self.heads * self.group
        x = self.proj.double().numpy()
        at = np.where(self.req >= 0, self.lengths[np.maximum(self.req, 0)] + self.pos, 0)
        turns = np.zeros(0, np.uint64) if turns is None else turns
        out = {}
        for name, part in (("k", x[:, hq:hq + self.heads]), ("v", x[:, hq + self.heads:])):
            c, s = self.codes[name].copy(), self.scale[name].copy()
            z = ref.rotate(part, at, turns, mscale, inter) if name == "k" else part
            out["blocks"] = ref.append(c, s, z, self.req, self.pos, self.lengths, self.table)
            out[name], out[name + "s"], out[name + "x"] = c, s, z
            out[name + "tol"] = ref.rotate_bound(part, len(turns), mscale, inter)
        out["q"] = ref.rotate(x[:, :hq], at, turns, mscale, inter)
        out["qtol"] = ref.rotate_bound(x[:, :hq], len(turns), mscale, inter)
        return out


CASES = [
    # w, lengths, heads, group, dim, page, dtype
    ([1], [0], 1, 1, 64, 16, "bf16"),
    ([16], [1000], 8, 4, 128, 16, "bf16"),
    ([1, 8, 3, 5], [15, 16, 17, 127], 2, 3, 64, 16, "f32"),
    ([4, 1, 7], [0, 31, 30], 3, 1, 48, 32, "bf16"),
    ([300], [0], 2, 2, 64, 64, "f32"),
    ([129, 2], [127, 128], 1, 4, 128, 128, "bf16"),
    ([0, 3, 0], [5, 5, 0], 2, 2, 256, 16, "bf16"),
    ([2] * 40, list(range(40)), 2, 1, 128, 16, "bf16"),
    # prompts: many rows in a block, teams of warps; heads that fill no team, or half of one
    ([40], [70], 3, 2, 128, 32, "bf16"),
    ([33, 34, 64], [0, 61, 63], 5, 1, 64, 64, "f32"),
    ([70, 0, 60], [9, 9, 100], 4, 2, 96, 64, "bf16"),
    # thousands of rows
    ([4100, 3], [5, 30], 2, 1, 64, 16, "bf16"),
    ([200, 4000, 1], [77, 0, 64], 1, 2, 128, 64, "bf16"),
    ([4097], [100], 1, 1, 128, 128, "f32"),
    ([2100, 2100], [0, 127], 2, 1, 48, 128, "bf16"),
]


@gpu
@pytest.mark.parametrize("case", CASES)
def test_append_without_rotation_is_exact(lib, case):
    w, lengths, heads, group, dim, page, dt = case
    c = Case(len(w) + dim, w, lengths, heads, group, dim, page, dt)
    got, want = c.run(None), c.want()
    for name in ("k", "v", "ks", "vs"):
        np.testing.assert_array_equal(got[name], want[name], err_msg=name)
    live = c.req >= 0
    np.testing.assert_array_equal(got["q"][live], want["q"][live])
    assert (got["q"][~live] == 9.0).all() and got["status"] == 0
    again = c.run(None, times=2)             # the same call once more leaves the same cache
    for name in ("k", "v", "ks", "vs"):
        np.testing.assert_array_equal(again[name], got[name], err_msg=name)


@gpu
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("inter", [False, True])
def test_append_with_rotation(lib, case, inter):
    w, lengths, heads, group, dim, page, dt = case
    c = Case(len(w) + dim + 1, w, lengths, heads, group, dim, page, dt)
    rot = dim if inter else dim // 2 // 16 * 16 or dim
    turns, mscale = bd.rope_turns(rot, 10000.0), 1.125
    rope = bd.Rope(torch.as_tensor(turns.view(np.int64)).cuda(), mscale, inter)
    got, want = c.run(rope), c.want(turns, mscale, inter)
    assert got["status"] == 0
    np.testing.assert_array_equal(got["v"], want["v"])
    np.testing.assert_array_equal(got["vs"], want["vs"])
    live = c.req >= 0
    tol = want["qtol"] + torch.finfo(c.dtype).eps / 2 * (np.abs(want["q"]) + want["qtol"])
    assert (np.abs(got["q"] - want["q"]) <= tol)[live].all()
    # no block's largest element may sit within the rotation's error of a power-of-two step
    touched = np.zeros(c.codes["k"].shape[0], bool)
    for p, rows in want["blocks"].items():
        touched[p] = True
        slots, rr = [s for s, _ in rows], [r for _, r in rows]
        for h in range(heads):
            amax = np.abs(want["kx"][rr, h]).max()
            frac = np.log2(amax / 448.0) % 1.0
            assert min(frac, 1 - frac) > 1e-5
            s = want["ks"][p, h]
            assert got["ks"][p, h] == s
            first = min(slots)
            np.testing.assert_array_equal(got["k"][p, h, :first], want["k"][p, h, :first])
            y = want["kx"][rr, h] / s
            t = want["ktol"][rr, h] / s
            d = np.abs(ref.decode(got["k"][p, h, slots]) - y)
            assert (d <= ref.half_step(np.abs(y) + t) + t).all()
            rest = np.setdiff1d(np.arange(first, page), slots)        # stale slots stay
            np.testing.assert_array_equal(got["k"][p, h, rest], c.codes["k"][p, h, rest])
    np.testing.assert_array_equal(got["k"][~touched], c.codes["k"][~touched])
    np.testing.assert_array_equal(got["ks"][~touched], c.scale["k"][~touched])


@gpu
def test_retained_codes_follow_a_growing_scale(lib):
    """Eight steps into one page, each 8 times larger than the last: codes are requantised step by
    step, and a step smaller than the page's scale leaves it alone."""
    dev = torch.device("cuda:0")
    table = torch.zeros(1, 1, dtype=torch.int32, device=dev)
    cache = bd.PagedCache.empty(1, 1, 16, 64, table)
    codes = {x: np.zeros((1, 1, 16, 64), np.uint8) for x in "kv"}
    scale = {x: np.ones((1, 1), np.float32) for x in "kv"}
    rng = np.random.default_rng(3)
    req, pos = np.zeros(2, np.int32), np.arange(2, dtype=np.int32)
    for step in range(8):
        size = 8.0 ** (step if step != 5 else 0)
        x = torch.as_tensor(rng.standard_normal((2, 2, 64)) * size).float()
        n = np.array([2 * step], np.int32)
        bd.dspark_append(cache, x[:, :1].to(dev), x[:, 1:].to(dev), torch.as_tensor(req).to(dev),
                         torch.as_tensor(pos).to(dev), torch.as_tensor(n).to(dev))
        for i, name in enumerate("kv"):
            ref.append(codes[name], scale[name], x[:, i:i + 1].double().numpy(), req, pos, n,
                       np.zeros((1, 1), int))
        np.testing.assert_array_equal(cache.k.view(torch.uint8).cpu().numpy(), codes["k"])
        np.testing.assert_array_equal(cache.v.view(torch.uint8).cpu().numpy(), codes["v"])
        np.testing.assert_array_equal(cache.k_scale.cpu().numpy(), scale["k"])
    assert scale["k"][0, 0] > 8.0 ** 7 / 448


@gpu
def test_values_at_the_ends_of_the_range(lib):
    """Zeros, the type's largest values, values under the smallest scale, infinities and NaN."""
    c = Case(1, [3, 2, 2, 1], [0, 16, 5, 0], 1, 1, 64, 16, "f32", spread=0.0)
    c.proj[0:3] = 0.0                                        # a block of zeros
    c.proj[3:5] = torch.finfo(torch.float32).max
    c.proj[5:7] *= 2.0 ** -100
    c.proj[7, :, ::2] = float("nan")
    c.proj[7, :, 1] = float("-inf")
    got, want = c.run(None), c.want()
    for name in ("k", "v", "ks", "vs"):
        np.testing.assert_array_equal(got[name], want[name], err_msg=name)
    assert got["status"] == bd.STATUS_BAD_VALUE
    assert got["ks"][c.table[0, 0], 0] == 2.0 ** -64 and got["ks"][c.table[1, 1], 0] == 2.0 ** 120


@gpu
def test_rows_and_pages_out_of_range_are_dropped(lib):
    c = Case(2, [2, 2, 2, 2, 1], [3, 3, 3, 3, 3], 2, 1, 64, 16, "bf16")
    base = c.want()
    c.table[1, 0] = c.n                      # past the pages
    c.table[2, 0] = -5
    c.lengths[3] = -1
    c.req[8] = 99                            # a request past B
    got = c.run(None)
    assert got["status"] == bd.STATUS_BAD_PAGE | bd.STATUS_BAD_LENGTH | bd.STATUS_BAD_ROWS
    p = c.table[0, 0]
    np.testing.assert_array_equal(got["k"][p], base["k"][p])
    others = np.arange(c.n) != p
    np.testing.assert_array_equal(got["k"][others], c.codes["k"][others])
    np.testing.assert_array_equal(got["v"][others], c.codes["v"][others])
    # a token past the table's width
    c = Case(2, [4], [14], 2, 1, 64, 16, "bf16")
    c.table = np.ascontiguousarray(c.table[:, :1])
    got = c.run(None)
    assert got["status"] == bd.STATUS_BAD_PAGE
    others = np.arange(c.n) != c.table[0, 0]
    np.testing.assert_array_equal(got["k"][others], c.codes["k"][others])
    assert (got["k"][c.table[0, 0], :, 14:] != c.codes["k"][c.table[0, 0], :, 14:]).any()


@gpu
def test_append_without_queries_and_on_another_stream(lib):
    c = Case(4, [5, 3], [10, 0], 2, 2, 128, 16, "bf16")
    want = c.want()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = c.run(None, with_q=False)
    np.testing.assert_array_equal(got["k"], want["k"])
    assert (got["q"] == 9.0).all()
