"""dspark_attend_shared against 64 bits over every request's whole context: one group and several, few
rows and many on either side of the prefix, prefixes of one page to many tiles and ends inside a tile;
groups that make no sense attend alone; pages out of range, queries that are no numbers, strides,
graphs, two calls in a row; the refusals.

Prefixes are computed apart only where that saves 6000 tiles of 128 tokens and a head: `heavy` adds a
group of 64 single tokens behind a prefix that is long enough for it, so that the others' odd sizes
are met in that form too."""
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

    def call(q=4096, hq=4, rows=3, B=2, gcu=4096, prefix=4096, groups=1, ws=4096, wb=1 << 30, scale=0.1):
        rc = lib.dspark_attend_shared(ctypes.byref(c), P(q), 256, P(4096), 256, hq, 0, rows, P(4096), P(4096), B,
                                      P(gcu), P(prefix), groups, scale, P(None), P(ws), wb, None, None)
        return rc, bd.last_error()

    need = bd.dspark_attend_shared_workspace_bytes(3, 4, 2, 64, 2)
    assert need == bd.dspark_attend_workspace_bytes(2, 64) + 3 * 4 * 65 * 4 + 12
    for code, kw, word in [(-1, dict(groups=-1), "groups"), (-1, dict(gcu=None), "group_cu"),
                           (-1, dict(prefix=None), "prefix"), (-1, dict(gcu=4097), "group_cu"),
                           (-1, dict(wb=need - 1), "workspace"), (-1, dict(ws=4104), "workspace"),
                           (-1, dict(ws=None), "workspace"), (-1, dict(hq=3), "q_heads"),
                           (-1, dict(q=None), "required"), (-1, dict(scale=float("inf")), "scale")]:
        rc, msg = call(**kw)
        assert rc == code and msg.startswith("dspark_attend_shared") and word in msg, (kw, rc, msg)
    assert call(rows=0, q=None)[0] == 0 and call(B=0)[0] == 0
    for bad in ((-1, 4, 2, 64, 2), (3, 3, 2, 64, 2), (3, 4, 2, 24, 2), (3, 4, 2, 64, -1), (3, 0, 1, 64, 2)):
        assert bd.dspark_attend_shared_workspace_bytes(*bad) == 0 and "bad sizes" in bd.last_error()


class Shared(Case):
    """groups: (requests, prefix) of consecutive groups from request 0 on; own: tokens of each request
    after its prefix."""

    def __init__(self, seed, w, own, groups, heads, group, dim, page, heavy=True, **kw):
        w, own, groups = list(w), list(own), list(groups)
        self.light = len(w)
        if heavy:
            tiles = -(-6000 // (63 * heads))
            w, own, groups = w + [1] * 64, own + [i % 5 for i in range(64)], groups + [(64, 128 * tiles)]
        # pages for the prefix of a group's first request and for every request's own tokens
        front, leads = np.zeros(len(w), np.int64), np.arange(len(w))
        b = 0
        for n, p in groups:
            front[b:b + n], leads[b:b + n] = p, b
            b += n
        mine = np.where(leads == np.arange(len(w)), front, 0)
        super().__init__(seed, w, mine + np.asarray(own), heads, group, dim, page, **kw)
        first = self.table
        self.table = np.full((len(w), first.shape[1] + int(front.max()) // page), -7, np.int32)
        for b in range(len(w)):
            at, skip = front[b] // page, mine[b] // page
            self.table[b, :at] = first[leads[b], :at]
            self.table[b, at:at + first.shape[1] - skip] = first[b, skip:]
        self.lengths = (front + np.asarray(own)).astype(np.int32)
        self.group_cu = np.cumsum([0] + [n for n, _ in groups]).astype(np.int32)
        self.prefix = np.asarray([p for _, p in groups], np.int32)

    def go(self, dtype, *, strides=False, prepare=False, lse=True, fill=0xAA):
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
        size = bd.dspark_attend_shared_workspace_bytes(self.rows, self.hq, self.heads, self.dim, len(self.lengths))
        ws = torch.full((size,), fill, dtype=torch.uint8, device=dev)
        cu, lengths, gcu, prefix = t(self.cu), t(self.lengths), t(self.group_cu), t(self.prefix)
        call = bd.dspark_attend_shared(cache, q, out, cu, lengths, gcu, prefix, ws, lse=ls, status=st, prepare=True)
        if prepare:
            return call, q, out, ls, (cache, ws, cu, lengths, gcu, prefix, st)
        call()
        call()                               # the second call finds the first's workspace
        torch.cuda.synchronize()
        return q.double().cpu().numpy(), out.double().cpu().numpy(), \
            ls.double().cpu().numpy() if lse else None, int(st.item())

    def hold(self, dtype=torch.bfloat16, status=0, **kw):
        q, out, lse, st = self.go(dtype, **kw)
        assert st == status
        forms_ref.check(self, dtype, q, out, lse, lambda b, pos: np.arange(pos + 1), joined=True)
        return out, lse


# w, own tokens, groups, heads, group, dim, page: the prefix's rows are few (the narrow kernel) or many
# (the wide one), the own tokens' too; prefixes that end inside a tile and at its end; cut over many CTAs
SHAPES = [
    ([1, 1], [0, 0], [(2, 16)], 1, 1, 64, 16),
    ([1, 1, 1], [0, 5, 130], [(3, 128)], 2, 4, 128, 128),
    ([4, 4, 4, 4], [20, 33, 60, 0], [(4, 992)], 2, 4, 128, 16),
    ([1] * 40, list(range(0, 400, 10)), [(40, 1024)], 2, 4, 128, 32),
    ([3, 1, 7, 2, 5], [1, 300, 0, 129, 15], [(2, 48), (3, 640)], 2, 3, 64, 16),
    ([2, 0, 3, 1, 0], [9, 50, 0, 700, 3], [(5, 5008)], 1, 8, 64, 16),
    ([1, 8] * 12, [7 * i for i in range(24)], [(6, 96), (10, 2048), (8, 320)], 1, 4, 128, 32),
    ([90, 60], [100, 3], [(2, 256)], 1, 4, 64, 64),
    ([40, 1, 70], [0, 900, 200], [(3, 3008)], 2, 2, 128, 64),
    ([16, 16], [2500, 1], [(2, 64)], 2, 2, 128, 64),
    ([1] * 4, [1] * 4, [(4, 9984)], 2, 2, 128, 128),
]


@gpu
@pytest.mark.parametrize("shape", SHAPES)
def test_shared(lib, shape):
    c = Shared(len(shape[0]) + shape[6], *shape)
    c.hold()
    c.q *= 5.0                               # one token takes nearly all, before or behind the prefix's end
    c.hold()


@gpu
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[4], SHAPES[7]])
@pytest.mark.parametrize("reach", [0, 100000])
def test_not_worth_it(lib, shape, reach):
    """Small calls attend alone, said by the host (a narrow page table) or on the device."""
    c = Shared(11, *shape, heavy=False)
    if reach:
        c.table = np.concatenate([c.table, np.full((len(c.lengths), reach // c.page), -7, np.int32)], 1)
    out, lse = c.hold()
    dev = torch.device("cuda:0")
    t = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(dev)         # noqa: E731
    cache = bd.PagedCache(t(c.codes["k"]), t(c.codes["v"]), t(c.scale["k"]), t(c.scale["v"]), t(c.table))
    q = torch.as_tensor(c.q).to(torch.bfloat16).to(dev)
    want = torch.full_like(q, 5.0)
    ws = torch.zeros(bd.dspark_attend_workspace_bytes(c.heads, c.dim), dtype=torch.uint8, device=dev)
    bd.dspark_attend(cache, q, want, t(c.cu), t(c.lengths), ws)
    np.testing.assert_array_equal(out, want.double().cpu().numpy())


@gpu
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[4]])
def test_fp32_attends_alone(lib, shape):
    Shared(1, *shape, heavy=False).hold(torch.float32)


@gpu
@pytest.mark.parametrize("dim", [16, 96, 256])
def test_other_head_sizes(lib, dim):
    for dtype in BOTH:
        Shared(dim, [3, 1], [40, 7], [(2, 64)], 2, 3, dim, 16, heavy=False).hold(dtype)


def base(seed=2):
    return Shared(seed, [2, 3, 1, 4, 2], [30, 5, 200, 64, 0], [(3, 160), (2, 320)], 2, 4, 128, 16)


@gpu
def test_a_prefix_counts_in_whole_pages(lib):
    c = base()
    want = c.go(torch.bfloat16)
    c.prefix += 15
    got = c.hold()
    np.testing.assert_array_equal(got[0], want[1])


@gpu
@pytest.mark.parametrize("what", ["one", "none", "short", "negative", "long", "gap", "outside", "backwards", "rows",
                                  "empty"])
def test_groups_that_attend_alone(lib, what):
    """Whatever the groups say, a row sees its request's tokens."""
    c = base(3)                              # groups of 3, 2 and 64 requests; 12 rows, then 64
    every = lambda b, pos: np.arange(pos + 1)                              # noqa: E731
    if what == "one":                        # groups of one request
        c.group_cu = np.concatenate([np.arange(6), [69]]).astype(np.int32)
        c.prefix = np.concatenate([[160] * 3, [320] * 2, c.prefix[2:]]).astype(np.int32)
    elif what == "none":
        c.prefix[:2] = 0
    elif what == "short":                    # a request with fewer tokens than the prefix
        c.lengths[1], c.lengths[20] = 100, 0
    elif what == "negative":
        c.prefix[:2] = [-16, -(1 << 31)]
    elif what == "long":                     # past the page table
        c.prefix[:2] = [1 << 30, 2 ** 31 - 1]
    elif what == "gap":                      # requests before, between and behind the groups
        c.group_cu[:3] = [1, 3, 3]
        c.group_cu[2:] = [5, 60]
        c.prefix[:2] = [160, 0]
    elif what == "outside":                  # requests that are none
        c.group_cu[3] = 70
        c.prefix[1] = 320
    elif what == "backwards":                # the first and second group are empty or nonsense
        c.group_cu[:3] = [3, 0, 5]
        c.prefix[:2] = [160, 64]
        c.table[3:5, :4] = c.table[0, :4]    # requests 0 to 4 now share 64 tokens
    elif what == "rows":                     # packed rows that end behind the buffer
        c.cu[69] = c.rows + 3
        q, out, lse, st = c.go(torch.bfloat16)
        assert st == bd.STATUS_BAD_ROWS
        c.cu[69] = c.cu[68]                  # the last request got nothing written
        forms_ref.check(c, torch.bfloat16, q, out, lse, every, joined=True)
        return
    elif what == "empty":                    # no rows in the first group; then no groups at all
        c = Shared(4, [0, 0, 2, 3], [30, 5, 200, 64], [(2, 160), (2, 320)], 2, 4, 64, 16)
        c.hold()
        c.group_cu, c.prefix = np.zeros(1, np.int32), np.zeros(0, np.int32)
    c.hold()


@gpu
def test_rows_of_no_request_inside_a_group(lib):
    """A request of a shared group whose rows run backwards is not written; the others are, whole."""
    c = base(12)
    c.cu[1:3] = [6, 5]                       # request 0: rows 0 .. 5, more than its pages hold; request 1: none
    q, out, lse, st = c.go(torch.bfloat16)
    assert st == bd.STATUS_BAD_ROWS | bd.STATUS_BAD_PAGE
    c.cu[1:3] = [5, 5]                       # row 5 is request 0's and request 2's
    want = forms_ref.attend(c, q, c.dim ** -0.5, lambda b, pos: np.arange(pos + 1))[0]
    np.testing.assert_allclose(out[:5], want[:5], atol=0.02, rtol=0.02)
    np.testing.assert_allclose(out[6:76], want[6:76], atol=0.02, rtol=0.02)


@gpu
def test_rows_that_are_more_than_there_are(lib):
    """Where cu_seqlens runs backwards, groups' rows may overlap: no group is then computed apart, and the
    rows of one request only are whole."""
    c = base(13)                             # 12 rows of requests 0 to 4, 64 of 5 to 68
    c.cu[3] = 60                             # request 2: rows 5 .. 59, more than its pages hold; request 3: none
    q, out, lse, st = c.go(torch.bfloat16)
    assert st == bd.STATUS_BAD_ROWS | bd.STATUS_BAD_PAGE
    c.cu[3:5] = [5, 10]                      # for the formula: request 2 none; 3 rows 5 .. 9, not looked at
    want = forms_ref.attend(c, q, c.dim ** -0.5, lambda b, pos: np.arange(pos + 1))[0]
    for rows in (slice(0, 5), slice(60, 76)):
        np.testing.assert_allclose(out[rows], want[rows], atol=0.02, rtol=0.02)
    assert (out[76:] == 5.0).all()


@gpu
@pytest.mark.parametrize("form", ["plain", "sinks", "shared"])
@pytest.mark.parametrize("rows,hq,page", [(2048, 64, 64), (200, 8, 128)])
def test_rows_that_overlap_without_end(lib, form, rows, hq, page):
    """Every other request has all the rows, over so many tokens that the work passes 32 bits: nothing is
    written."""
    B, dim, width = 1024, 64, 32768
    dev = torch.device("cuda:0")
    z = lambda *s, **k: torch.zeros(*s, device=dev, **k)                   # noqa: E731
    cu = torch.tensor([0, rows] * (B // 2) + [rows], dtype=torch.int32, device=dev)
    table = z(B, width, dtype=torch.int32)
    reach = width * page
    codes = [z(4, 1, page, dim, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.ones(4, 1, device=dev) for _ in range(2)]
    cache = bd.PagedCache(*codes, *scales, table)
    lengths = torch.full((B,), reach - rows, dtype=torch.int32, device=dev)
    q = z(rows, hq, dim, dtype=torch.bfloat16)
    out = torch.full_like(q, 5.0)
    st = z(1, dtype=torch.int32)
    if form == "shared":
        ws = z(bd.dspark_attend_shared_workspace_bytes(rows, hq, 1, dim, B), dtype=torch.uint8)
        gcu, prefix = (torch.tensor(x, dtype=torch.int32, device=dev) for x in ([0, B], [100 * page]))
        bd.dspark_attend_shared(cache, q, out, cu, lengths, gcu, prefix, ws, status=st)
    else:
        ws = z(bd.dspark_attend_workspace_bytes(1, dim), dtype=torch.uint8)
        if form == "plain":
            bd.dspark_attend(cache, q, out, cu, lengths, ws, status=st)
        else:
            bd.dspark_attend_sinks(cache, q, out, cu, lengths, ws, window=reach, sinks=4, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == bd.STATUS_BAD_ROWS
    assert bool((out == 5.0).all())


@gpu
def test_bad_pages(lib):
    c = base(5)
    c.table[:3, 4] = c.n                     # in the first prefix
    c.table[3:5, 0] = -1
    c.table[2, 17] = 10 ** 6                 # one of request 2's own
    c.hold(status=bd.STATUS_BAD_PAGE)
    c = Shared(6, [2, 1, 70], [0, 0, 20], [(3, 64)], 1, 4, 64, 64)
    c.table[:3, 0] = -1                      # nothing of the prefix: the own tokens alone
    out, lse = c.hold(status=bd.STATUS_BAD_PAGE)
    c.table[:3] = -1                         # nothing at all
    _, lse = c.hold(status=bd.STATUS_BAD_PAGE)
    assert np.isneginf(lse[:73]).all()


@gpu
def test_queries_that_are_no_numbers(lib):
    c = base(7)
    _, clean, _, _ = c.go(torch.bfloat16)
    c.q[2, 1, 5], c.q[7, 2, 0] = np.nan, np.inf
    _, out, _, _ = c.go(torch.bfloat16)
    hit = np.zeros(out.shape[:2], bool)
    hit[2, 1] = hit[7, 2] = True
    assert np.isnan(out[hit]).all()
    np.testing.assert_array_equal(out[~hit], clean[~hit])


@gpu
@pytest.mark.parametrize("shape", [SHAPES[3], SHAPES[8]])
def test_strides_no_lse_and_the_same_bits(lib, shape):
    c = Shared(8, *shape)
    out, _ = c.hold()
    for kw in (dict(strides=True), dict(lse=False), dict(fill=0xFF)):
        np.testing.assert_array_equal(c.go(torch.bfloat16, **kw)[1], out)


@gpu
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[8]])
def test_graph_on_another_stream(lib, shape):
    """Replays with other groups in the same buffers too."""
    c = Shared(9, *shape)
    want = c.go(torch.bfloat16)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call, q, out, lse, keep = c.go(torch.bfloat16, prepare=True)
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
    keep[5].fill_(c.page)                    # a prefix of one page
    graph.launch()
    torch.cuda.synchronize()
    forms_ref.check(c, torch.bfloat16, q.double().cpu().numpy(), out.double().cpu().numpy(),
                    lse.double().cpu().numpy(), lambda b, pos: np.arange(pos + 1), joined=True)


@gpu
@pytest.mark.parametrize("seed", range(10))
def test_random_shapes(lib, seed):
    rng = np.random.default_rng(500 + seed)
    G = int(rng.integers(1, 5))
    page = int(rng.choice([16, 32, 64, 128]))
    groups = [(int(rng.integers(1, 7)), int(rng.integers(0, 900)) // page * page) for _ in range(G)]
    B = sum(n for n, _ in groups)
    w = rng.integers(0, 9, B) if seed % 3 else rng.integers(0, 60, B)
    w[0] = max(w[0], 1)
    Shared(seed, w, rng.integers(0, 500, B), groups, int(rng.integers(1, 4)), int(rng.integers(1, 9)),
           int(rng.choice([64, 128])), page, spread=2.0).hold()
