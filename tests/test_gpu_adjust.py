"""dspark_adjust against the formula in 64 bits: both types, vocabularies of one token to many
slices, rows at every alignment, in place and not, histories, drafts, biases (one token several
times), grammar masks (shared rows, none, empty ones), values that are no numbers in masked places;
rows of no request; what is out of range; streams, graphs, offsets past 32 bits; the refusals.

Tolerance: at most four roundings to fp32 on the way (quotient, penalty, difference, bias), each
2^-24 of the largest magnitude met, and one rounding to the type."""
import ctypes

import numpy as np
import pytest
import torch

from speculative_decoding_ragged_gb300 import _binding as bd

gpu = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_ragged_gb300 import build
    build.build()
    return bd.lib()


def test_refuses_on_the_host(lib):
    P = ctypes.c_void_p

    def call(how="given", x=4096, xs=100, y=8192, ys=100, dt=0, rows=6, V=100, cu=4096, tok=4096,
             B=2, gamma=3, **h):
        c = bd._Adjustments()
        for name, value in h.items():
            setattr(c, name, value)
        rc = lib.dspark_adjust(P(x), xs, P(y), ys, dt, rows, V, P(cu), P(tok), B, gamma,
                               ctypes.byref(c) if how == "given" else None, None, None)
        return rc, bd.last_error()

    mask = dict(mask=4096, mask_stride=4, mask_rows=6)
    for code, kw, word in [
            (-1, dict(how=None), "how"), (-1, dict(dt=7), "dtype"), (-1, dict(rows=-1), "rows=-1"),
            (-1, dict(V=0), "V=0"), (-1, dict(B=-1), "B=-1"), (-1, dict(gamma=0), "gamma=0"),
            (-1, dict(gamma=33), "gamma=33"), (-2, dict(B=8193), "B = 8193"),
            (-2, dict(V=2 ** 29, xs=1 << 30, ys=1 << 30), "V = "),
            (-1, dict(xs=99), "row strides"), (-1, dict(ys=99), "row strides"),
            (-1, dict(y=4096, ys=101), "in place"), (-1, dict(cu=None, rows=5), "cu_seqlens"),
            (-1, dict(history_cap=-1), "history_cap"), (-2, dict(history_cap=524001), "history_cap"),
            (-1, dict(history=4096), "history_len"),
            (-1, dict(bias_tokens=4096), "bias"), (-2, dict(bias_tokens=4096, bias_cap=2048), "bias_cap"),
            (-1, dict(mask=4096, mask_stride=3, mask_rows=6), "mask"),
            (-1, dict(mask=4096, mask_stride=4, mask_rows=5), "mask_row"),
            (-1, dict(x=None), "required"), (-1, dict(y=None), "required"),
            (-1, dict(y=8193), "aligned"), (-1, dict(tok=None, repetition=4096), "block_tokens"),
            (-1, dict(tok=4098), "4-byte"), (-1, dict(mask, mask_row=4097), "4-byte")]:
        rc, msg = call(**kw)
        assert rc == code and msg.startswith("dspark_adjust") and word in msg, (kw, rc, msg)
    assert call(rows=0, x=None, y=None, V=1)[0] == 0 and call(B=0, cu=None, rows=0)[0] == 0


def test_binding_refuses():
    i = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="go together"):
        bd.Adjustments(history=i)
    with pytest.raises(ValueError, match="go together"):
        bd.Adjustments(bias_tokens=i)
    with pytest.raises(ValueError, match="needs a mask"):
        bd.Adjustments(mask_row=i[0])
    with pytest.raises(ValueError, match="CUDA"):
        bd.Adjustments(repetition=torch.ones(2))
    with pytest.raises(ValueError, match="words"):
        bd.Adjustments(mask=i.float())


class Case:
    """B requests with windows w; everything a call may be given, as numpy arrays."""

    def __init__(self, seed, w, V, cap=60, n_bias=12, pad=3, gamma=None, masks=5):
        rng = np.random.default_rng(seed)
        self.rng = rng
        self.w, self.V, B = list(w), V, len(w)
        self.gamma = gamma or max(max(w), 1)
        self.cu = np.concatenate([[0], np.cumsum(w)]).astype(np.int32)
        self.rows = int(self.cu[-1]) + pad
        self.x = rng.standard_normal((self.rows, V)) * 3
        tok = lambda *s: (V * rng.random(s) ** 3).astype(np.int32)          # noqa: E731
        self.blocks = tok(B, self.gamma)
        self.h = dict(history=tok(B, cap), history_len=rng.integers(0, cap + 1, B).astype(np.int32))
        self.h["history_len"][: 2] = [0, cap][: min(2, B)]
        self.h["prompt_len"] = (self.h["history_len"] * rng.random(B)).astype(np.int32)
        if cap > 8:
            self.h["history"][B - 1, 3:] = self.h["history"][B - 1, 3]      # one token again and again
        self.h["repetition"] = rng.uniform(0.7, 1.6, B).astype(np.float32)
        self.h["presence"] = rng.uniform(-0.5, 1.0, B).astype(np.float32)
        self.h["frequency"] = rng.uniform(-0.2, 0.6, B).astype(np.float32)
        if n_bias:
            self.h["bias_tokens"] = tok(B, n_bias)                          # some token several times
            self.h["bias_values"] = (rng.standard_normal((B, n_bias)) * 5).astype(np.float32)
            self.h["bias_values"][rng.random((B, n_bias)) < 0.15] = -np.inf
            self.h["bias_len"] = rng.integers(0, n_bias + 1, B).astype(np.int32)
        if masks:
            words = -(-V // 32)
            bits = rng.random((masks, V)) < rng.choice([0.02, 0.5, 0.98], masks)[:, None]
            bits[np.arange(masks), rng.integers(0, V, masks)] = True
            full = np.ones((masks, words * 32), bool)                       # bits past V: set
            full[:, :V] = bits
            self.h["mask"] = np.packbits(full, axis=1, bitorder="little").view("<u4").view(np.int32)
            self.h["mask_row"] = rng.integers(-1, masks, self.rows).astype(np.int32)

    def without(self, *names):
        for n in names:
            self.h.pop(n, None)
        return self

    def want(self, x):
        """The formula in 64 bits on x [rows, V] (as held by the device): results, and the largest
        magnitude met on the way, for the rows of requests; which rows those are."""
        h, V = self.h, self.V
        y, big = x.astype(np.float64).copy(), np.abs(x.astype(np.float64))
        mine = np.zeros(self.rows, bool)
        for b, w in enumerate(self.w):
            get = lambda n, d: float(h[n][b]) if n in h else d              # noqa: E731
            rep, pres, freq = get("repetition", 1.0), get("presence", 0.0), get("frequency", 0.0)
            n = int(h["history_len"][b]) if "history" in h else 0
            p = int(h["prompt_len"][b]) if "prompt_len" in h else 0
            ids = h["history"][b, :n] if "history" in h else np.zeros(0, int)
            count = lambda a: np.bincount(a, minlength=V)[:V]               # noqa: E731
            bias = {}
            if "bias_tokens" in h:
                for t, v in zip(h["bias_tokens"][b][:h["bias_len"][b]], h["bias_values"][b]):
                    bias[int(t)] = float(v)
            for i in range(w):
                r = self.cu[b] + i
                mine[r] = True
                uses = count(ids[p:]) + count(self.blocks[b, 1:i + 1])
                seen = (uses + count(ids[:p])) > 0
                with np.errstate(invalid="ignore"):
                    z = y[r]
                    z = np.where(seen, np.where(z > 0, z / rep, z * rep), z)
                    big[r] = np.maximum(big[r], np.abs(z))
                    off = np.where(uses > 0, freq * uses + pres, 0.0)
                    big[r] = np.maximum(big[r], np.abs(freq) * uses + abs(pres))
                    z = z - off
                    for t, v in bias.items():
                        z[t] += v
                        if np.isfinite(v):
                            big[r, t] = max(big[r, t], abs(v), abs(z[t]))
                    big[r] = np.maximum(big[r], np.where(np.isfinite(z), np.abs(z), 0))
                if "mask" in h:
                    m = h["mask_row"][r] if "mask_row" in h else r
                    if 0 <= m < len(h["mask"]):
                        bits = np.unpackbits(h["mask"][m].view(np.uint8), bitorder="little")[:V]
                        z[bits == 0] = -np.inf
                y[r] = z
        return y, big, mine

    def run(self, dtype, in_place=False, offset=0, extra=0, static=False, **more):
        dev = torch.device("cuda:0")
        t = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(dev)      # noqa: E731
        wide = torch.full((self.rows, self.V + extra + offset), 7.0, dtype=dtype, device=dev)
        x = wide[:, offset:offset + self.V]
        x.copy_(torch.as_tensor(self.x).to(dtype))
        if in_place:
            out = x
        else:
            out = torch.full((self.rows, self.V + extra), 9.0, dtype=dtype, device=dev)[:, :self.V]
        before, given = out.clone(), x.clone()
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        how = bd.Adjustments(**{k: t(v) for k, v in self.h.items()})
        blocks, cu = t(self.blocks), None if static else t(self.cu)
        call = bd.dspark_adjust(x, out, blocks, how, cu_seqlens=cu, status=status, prepare=True, **more)
        call()
        torch.cuda.synchronize()
        return dict(x=x, given=given, out=out, before=before, status=int(status.item()), call=call,
                    wide=wide, keep=(how, blocks, cu))

    def check(self, got, dtype):
        x = got["given"].float().cpu().numpy().astype(np.float64)
        want, big, mine = self.want(x)
        out = got["out"].float().cpu().numpy().astype(np.float64)
        before = got["before"].float().cpu().numpy()
        np.testing.assert_array_equal(out[~mine], before[~mine])
        out, want, big = out[mine], want[mine], big[mine]
        assert (np.isnan(out) == np.isnan(want)).all()
        inf = np.isinf(want)
        assert (out[inf] == want[inf]).all() and not np.isinf(out[~inf]).any()
        fine = np.isfinite(want)
        tol = 4 * 2.0 ** -24 * big[fine]
        tol = tol + HALF[dtype] * (np.abs(want[fine]) + tol) + 1e-38
        err = np.abs(out[fine] - want[fine])
        assert (err <= tol).all(), float((err - tol).max())
        same = np.isfinite(want) & (want == x[mine])
        assert (out[same] == want[same]).all()             # untouched logits keep their bits


# slices of 1024 tokens (few requests) to 7168 (304 requests and more); odd vocabularies put the rows
# at every alignment
@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("w,V", [([1], 1), ([3, 1], 31), ([2, 0, 4], 33), ([5, 2], 257), ([1, 8, 3], 1024),
                                 ([4, 1, 2], 4099), ([7], 20011), ([2, 3], 151936), ([2] * 310, 500),
                                 ([1, 2] * 80, 20001)])
def test_against_the_formula(lib, dtype, w, V):
    c = Case(V, w, V)
    got = c.run(dtype)
    c.check(got, dtype)
    assert got["status"] == 0


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset,extra", [(0, 0), (1, 0), (3, 5), (8, 8)])
@pytest.mark.parametrize("in_place", [False, True])
def test_places_and_strides(lib, dtype, offset, extra, in_place):
    c = Case(offset, [3, 5, 1], 2051)
    got = c.run(dtype, in_place=in_place, offset=offset, extra=extra)
    c.check(got, dtype)
    assert got["status"] == 0
    if offset:
        assert (got["wide"][:, :offset] == 7).all()
    if extra:
        assert (got["wide"][:, offset + c.V:] == 7).all()


# Batches large enough for the largest slices (7168 tokens); row strides are padded so that odd
# vocabularies' rows lie on 16-byte boundaries too.
LARGE = [([1] * 310, 1), ([2, 0, 1] * 110, 7), ([3, 1] * 160, 33), ([2] * 310, 515), ([1, 4] * 80, 7169),
         ([5, 2, 8] * 21, 40003), ([2] * 40, 60000)]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("w,V", LARGE)
def test_large_calls(lib, dtype, w, V):
    c = Case(V, w, V)
    got = c.run(dtype, extra=-V % 8)
    c.check(got, dtype)
    assert got["status"] == 0
    again = c.run(dtype, extra=-V % 8, in_place=True)       # the same bits in place
    M = int(c.cu[-1])
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
    assert torch.equal(got["out"][:M].contiguous().view(bits), again["out"][:M].contiguous().view(bits))


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("left_out", [("repetition", "presence", "frequency"), ("bias_tokens", "bias_values", "bias_len"),
                                      ("mask", "mask_row"), ("mask_row",),
                                      ("repetition", "presence", "frequency", "bias_tokens", "bias_values", "bias_len")])
def test_large_calls_without_parts(lib, dtype, left_out):
    c = Case(14, [2, 1] * 155, 3001, masks=470 if "mask_row" in left_out else 7).without(*left_out)
    c.x[c.rng.random(c.x.shape) < 0.05] = np.nan
    c.x[c.rng.random(c.x.shape) < 0.05] = -np.inf
    if "bias_values" in c.h:
        c.h["bias_values"][np.isinf(c.h["bias_values"])] = 1.0
    got = c.run(dtype, extra=-3001 % 8)
    c.check(got, dtype)
    assert got["status"] == 0


@gpu
def test_large_calls_with_forbidden_rows(lib):
    """Masks that forbid whole parts and whole rows, mask rows out of range, requests that are none."""
    c = Case(15, [2, 3] * 60, 20480, masks=6).without("bias_tokens", "bias_values", "bias_len")
    c.h["mask"][0] = 0
    c.h["mask"][1] = 0
    c.h["mask"][1, 639] = -1 << 31               # the last token alone
    c.h["mask"][2] = -1
    c.h["mask"][2, 32:64] = 0                    # one part of 1024 tokens
    c.h["mask"][3] = 0
    c.h["mask"][3, 31:33] = 1
    got = c.run(torch.bfloat16)
    c.check(got, torch.bfloat16)
    assert got["status"] == (bd.STATUS_NO_TOKEN if (c.h["mask_row"][:300] == 0).any() else 0)
    c.h["mask_row"][7] = 6
    c.cu[-1] += 100
    got = c.run(torch.bfloat16)
    assert got["status"] & bd.STATUS_BAD_ROWS
    assert torch.equal(got["out"][c.cu[-2]:], got["before"][c.cu[-2]:])


PENALTIES = ("repetition", "presence", "frequency")
HISTORY = ("history", "history_len", "prompt_len")
BIAS = ("bias_tokens", "bias_values", "bias_len")
MASK = ("mask", "mask_row")


@gpu
@pytest.mark.parametrize("left_out", [(), PENALTIES, HISTORY, BIAS, MASK, ("prompt_len",), ("repetition",),
                                      ("presence", "frequency"), PENALTIES + HISTORY + BIAS,
                                      PENALTIES + HISTORY + MASK, PENALTIES + HISTORY + BIAS + MASK])
@pytest.mark.parametrize("in_place", [False, True])
def test_parts_left_out(lib, left_out, in_place):
    c = Case(5, [3, 4, 2], 5003).without(*left_out)
    got = c.run(torch.bfloat16, in_place=in_place)
    c.check(got, torch.bfloat16)
    assert got["status"] == 0


@gpu
def test_neutral_penalties_change_nothing(lib):
    c = Case(6, [3, 2], 700).without(*BIAS, *MASK)
    for name, v in zip(PENALTIES, (1.0, 0.0, 0.0)):
        c.h[name][:] = v
    got = c.run(torch.bfloat16)
    assert torch.equal(got["out"][:5], got["given"][:5])


@gpu
def test_long_histories_and_the_same_token(lib):
    c = Case(7, [4, 2], 3001, cap=40000)
    c.h["history"][0] = 17
    c.h["history_len"][:] = [40000, 39999]
    c.h["prompt_len"][:] = [1, 39999]
    c.blocks[0, 1:] = 17
    got = c.run(torch.float32)
    c.check(got, torch.float32)
    assert got["status"] == 0


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_numbers(lib, dtype):
    """NaN and infinities: gone where masked, kept (through the formula) where allowed."""
    c = Case(8, [4, 4], 999)
    c.x[c.rng.random(c.x.shape) < 0.2] = np.nan
    c.x[c.rng.random(c.x.shape) < 0.1] = np.inf
    c.x[c.rng.random(c.x.shape) < 0.1] = -np.inf
    c.h["bias_values"][np.isinf(c.h["bias_values"])] = 1.0         # inf - inf is tested apart
    got = c.run(dtype)
    c.check(got, dtype)


@gpu
def test_masks_that_allow_nothing(lib):
    c = Case(9, [3, 2], 3333, masks=4).without(*BIAS)
    c.h["mask"][1] = 0                        # none at all
    c.h["mask"][2] = 0
    c.h["mask"][2, -1] = -1 << (3333 % 32)    # bits past V only
    c.h["mask"][3] = 0
    c.h["mask"][3, 50] = 1 << 7               # one token
    c.h["mask_row"][:5] = [1, 2, 3, -1, 3]
    got = c.run(torch.bfloat16)
    c.check(got, torch.bfloat16)
    assert got["status"] == bd.STATUS_NO_TOKEN
    assert torch.isfinite(got["out"][2]).sum() == 1 and torch.isinf(got["out"][:2]).all()


@gpu
def test_a_mask_per_row(lib):
    c = Case(10, [3, 2], 100, masks=8, pad=3).without("mask_row")
    got = c.run(torch.float32)
    c.check(got, torch.float32)


@gpu
def test_static_rows(lib):
    c = Case(11, [4, 4, 4], 1111, gamma=4, pad=2)
    got = c.run(torch.bfloat16, static=True)
    c.check(got, torch.bfloat16)


@gpu
def test_out_of_range(lib):
    S = bd
    c = Case(12, [2, 3, 1], 500)
    good = {k: v.copy() for k, v in c.h.items()}

    def status(change, cu=None, blocks=None, check=True):
        c.h = {k: v.copy() for k, v in good.items()}
        change(c.h)
        keep = c.cu, c.blocks
        c.cu = keep[0] if cu is None else np.asarray(cu, np.int32)
        c.blocks = keep[1] if blocks is None else blocks
        got = c.run(torch.float32)
        c.cu, c.blocks = keep
        return got

    # tokens outside the vocabulary are left out: as a history without them
    got = status(lambda h: (h["history"].__setitem__((1, slice(0, 2)), [-5, 500]),
                            h["history_len"].__setitem__(1, 30), h["prompt_len"].__setitem__(1, 2)))
    assert got["status"] == S.STATUS_BAD_TOKEN
    a = got["out"]
    got = status(lambda h: (h["history"].__setitem__((1, slice(0, 28)), h["history"][1, 2:30]),
                            h["history_len"].__setitem__(1, 28), h["prompt_len"].__setitem__(1, 0)))
    assert got["status"] == 0 and torch.equal(a, got["out"])
    assert status(lambda h: (h["bias_tokens"].__setitem__((0, 0), 1 << 30),
                             h["bias_len"].__setitem__(0, 1)))["status"] == S.STATUS_BAD_TOKEN
    blocks = c.blocks.copy()
    blocks[1, 1] = -1
    assert status(lambda h: None, blocks=blocks)["status"] == S.STATUS_BAD_TOKEN
    blocks[1, 1], blocks[:, 0] = 3, 10 ** 9      # the anchor is the history's last: not looked at
    assert status(lambda h: None, blocks=blocks)["status"] == 0
    # lengths are clamped
    for name, bad in [("history_len", 61), ("history_len", -1), ("bias_len", 13), ("bias_len", -2)]:
        got = status(lambda h: h[name].__setitem__(1, bad))
        assert got["status"] == S.STATUS_BAD_LENGTH, name
        c.h[name][1] = min(max(bad, 0), 60 if name == "history_len" else 12)
        c.h["prompt_len"] = np.minimum(c.h["prompt_len"], c.h["history_len"])
        c.check(got, torch.float32)
    got = status(lambda h: h["prompt_len"].__setitem__(1, 61))
    assert got["status"] == S.STATUS_BAD_LENGTH
    # values
    for name, bad in [("repetition", 0.0), ("repetition", -1.0), ("repetition", np.nan),
                      ("presence", np.inf), ("frequency", np.nan)]:
        got = status(lambda h: h[name].__setitem__(1, bad))
        assert got["status"] == S.STATUS_BAD_VALUE, name
        c.h[name][1] = 1.0 if name == "repetition" else 0.0
        c.check(got, torch.float32)
    for bad in (np.nan, np.inf):
        got = status(lambda h: (h["bias_len"].__setitem__(1, 1), h["bias_values"].__setitem__((1, 0), bad)))
        assert got["status"] == S.STATUS_BAD_VALUE
        c.h["bias_len"][1] = 0
        c.check(got, torch.float32)
    # mask rows and rows
    for bad in (-2, 5, 1 << 30):
        got = status(lambda h: h["mask_row"].__setitem__(2, bad))
        assert got["status"] == S.STATUS_BAD_ROWS
        c.check(got, torch.float32)              # want() takes it as none
    for cu in ([0, 2, 5, 10], [-1, 2, 5, 6], [0, 2, 1, 2]):
        got = status(lambda h: None, cu=cu)
        assert got["status"] == S.STATUS_BAD_ROWS, cu
    c.gamma = 2                                  # request 1 has three rows
    got = status(lambda h: None, blocks=c.blocks[:, :2])
    assert got["status"] == S.STATUS_BAD_ROWS
    assert torch.equal(got["out"][2:5], got["before"][2:5])


@gpu
def test_other_streams_and_a_replayed_graph(lib):
    c = Case(13, [3, 1, 4], 6001)
    eager = c.run(torch.bfloat16)["out"].clone()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        got = c.run(torch.bfloat16)
        assert torch.equal(got["out"], eager)
        got["out"].fill_(9.0)
        graph = bd.StepGraph(stream)
        got["call"]()
        graph.end()
    stream.synchronize()
    assert (got["out"] == 9).all()
    for _ in range(2):
        graph.launch()
    torch.cuda.synchronize()
    assert torch.equal(got["out"], eager)
    got["x"].neg_()                              # new logits in the same buffer
    got["given"] = got["x"].clone()
    got["before"].fill_(9.0)
    graph.launch()
    torch.cuda.synchronize()
    c.check(got, torch.bfloat16)


@gpu
def test_offsets_past_32_bits(lib):
    """In place over more than 2^32 bytes: the last request's rows, checked alone."""
    dev = torch.device("cuda:0")
    V, gamma, B = 151936, 16, 900
    x = torch.zeros(B * gamma, V, dtype=torch.bfloat16, device=dev)
    assert x.numel() * 2 > 2 ** 32
    x[-2:] = 2.0
    history = torch.zeros(B, 4, dtype=torch.int32, device=dev)
    history[-1] = torch.tensor([5, 5, 9, V - 1])
    n = torch.full((B,), 4, dtype=torch.int32, device=dev)
    one = torch.ones(B, device=dev)
    mask = torch.full((B * gamma, -(-V // 32)), -1, dtype=torch.int32, device=dev)
    mask[-1, 0] = ~(1 << 3)
    how = bd.Adjustments(history=history, history_len=n, presence=one, frequency=one, mask=mask)
    blocks = torch.full((B, gamma), 9, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    bd.dspark_adjust(x, x, blocks, how, status=status)
    want = torch.full((V,), 2.0)
    want[5], want[9], want[V - 1], want[3] = 2 - 3, 2 - (1 + 16), 2 - 2, -float("inf")
    assert torch.equal(x[-1].float().cpu(), want)
    assert int(status.item()) == 0
