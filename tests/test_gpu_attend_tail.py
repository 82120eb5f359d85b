"""dspark_attend where one token holds much of a row's weight and a long tail of small weights the
rest, with values of its own near zero: what an attention sink looks like. The result is then the
tail's, so every small weight counts. Many requests read the same pages, which makes enough units
that no run's end cuts most of them: a run then holds the dominant token and its whole tail.

Tolerance, from the header: a weight is within 2^-8 of itself, so a result within 2^-8 of
sum p |v|; the scores as in test_gpu_attend (queries here are held exactly by their pieces); one
rounding to bf16. There is no term for weights under some share of the largest."""
import numpy as np
import pytest
import torch

from speculative_decoding_ragged_gb300 import _binding as bd

gpu = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_ragged_gb300 import build
    build.build()
    return bd.lib()


def quantise(x):
    """[n_pages, heads, page, dim] -> codes and power-of-two scales."""
    top = x.abs().amax(dim=(2, 3)).clamp(min=2.0 ** -40)
    scale = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
    return (x / scale[:, :, None, None]).float().to(FP8), scale.float()


class Sink:
    """B requests with the same pages and the same queries: `context` tokens and w rows. The tokens
    `at` hold about `share` of every row's weight."""

    def __init__(self, context, share, w, dim, group, flat, at=0, heads=4, B=80, page=64, seed=0):
        dev = torch.device("cuda:0")
        g = torch.Generator(device=dev).manual_seed(seed)
        self.B, self.w, self.dim, self.group, self.heads = B, w, dim, group, heads
        self.n = context + w
        blocks = -(-self.n // page)
        rand = lambda *s: torch.randn(*s, generator=g, device=dev, dtype=torch.float64)    # noqa: E731
        k = rand(heads, blocks * page, dim) * (0.0 if flat else 1.0)
        v = rand(heads, blocks * page, dim) * 0.5 + 1.0
        # magnitudes from 1/2 to 4: two pieces of 4 bits hold such queries' 8 bits
        q = torch.exp2(torch.rand(w, heads * group, dim, generator=g, device=dev, dtype=torch.float64) * 3 - 1)
        q = q * torch.sign(rand(w, heads * group, dim))
        q[..., 0] = 4.0
        self.q = q.to(torch.bfloat16)
        k[:, :, 0] = 0.0
        self.scale = dim ** -0.5
        s = torch.einsum("whgd,htd->hwgt", self.q.double().view(w, heads, group, dim), k) * self.scale
        # the dominant token's score, for a share of about `share` of the weight in every row
        at = [at] if isinstance(at, int) else list(at)
        want = torch.logsumexp(s, -1).mean() + np.log(share / len(at) / (1 - share))
        for t in at:
            k[:, t] = 0.0
            k[:, t, 0] = want / (4.0 * self.scale)
            v[:, t] = rand(heads, dim) * 1e-3
        paged = lambda x: x.view(heads, blocks, page, dim).transpose(0, 1).contiguous()    # noqa: E731
        self.k, self.ks = quantise(paged(k))
        self.v, self.vs = quantise(paged(v))
        self.table = torch.arange(blocks, dtype=torch.int32, device=dev).repeat(B, 1)
        self.context = context

    def run(self):
        dev = self.q.device
        cache = bd.PagedCache(self.k, self.v, self.ks, self.vs, self.table)
        q = self.q.repeat(self.B, 1, 1)
        out = torch.full_like(q, 5.0)
        lse = torch.zeros(q.shape[:2], device=dev)
        cu = (torch.arange(self.B + 1, device=dev) * self.w).to(torch.int32)
        lengths = torch.full((self.B,), self.context, dtype=torch.int32, device=dev)
        ws = torch.empty(bd.dspark_attend_workspace_bytes(self.heads, self.dim), dtype=torch.uint8, device=dev)
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        bd.dspark_attend(cache, q, out, cu, lengths, ws, lse=lse, status=st)
        assert int(st.item()) == 0
        return out.view(self.B, self.w, -1, self.dim).double(), lse.view(self.B, self.w, -1).double()

    def exact(self):
        """out, sum p |v|, lse, and the largest scale * sum |q k| of a row: [w, heads, ...]."""
        flat = lambda c, s: (c.double() * s.double()[:, :, None, None]).transpose(0, 1).reshape(   # noqa: E731
            self.heads, -1, self.dim)[:, :self.n]
        k, v = flat(self.k, self.ks), flat(self.v, self.vs)
        hide = torch.arange(self.n, device=k.device)[None] > \
            torch.arange(self.context, self.n, device=k.device)[:, None]
        q = self.q.double().view(self.w, self.heads, self.group, self.dim)
        outs = []
        for h in range(self.heads):
            s = torch.einsum("wgd,td->gwt", q[:, h], k[h]) * self.scale
            s = s.masked_fill(hide[None], float("-inf"))
            lse = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[..., None])
            big = torch.einsum("wgd,td->gwt", q[:, h].abs(), k[h].abs()).amax(-1) * self.scale
            outs.append([x.transpose(0, 1) for x in (p @ v[h], p @ v[h].abs(), lse, big, p.amax(-1))])
        return [torch.cat([o[i] for o in outs], 1) for i in range(5)]

    def check(self, out_too=True):
        out, got_lse = self.run()
        want, spread, lse, big, top = self.exact()
        ds = (self.dim + 8) * 2.0 ** -24 * big
        assert bool(((got_lse - lse).abs() <= 2 * ds + 2.0 ** -20 * (1 + lse.abs())).all())
        if not out_too:
            return top
        tol = spread * (torch.exp(2 * ds) - 1 + 2.0 ** -20 + 2.0 ** -8)[..., None]
        tol = tol + torch.finfo(torch.bfloat16).eps / 2 * (want.abs() + tol)
        err = (out - want[None]).abs()
        assert bool((err <= tol).all()), ("times the bound", float((err / tol).max()))
        return top


@gpu
@pytest.mark.parametrize("at", [0, (0, 130), (0, 1, 2, 3), (5, 3000)])
@pytest.mark.parametrize("w", [8, 40])
def test_log_sum_of_many_equal_weights(lib, w, at):
    """Equal addends round the same way every time: one fp32 sum over all tokens would drift."""
    Sink(131072, 0.95, w, 128, 4, True, at=at).check(out_too=False)


WINDOWS = [1, 4, 8, 40]                      # 4, 16, 32 and 160 (position, head) rows of a cache head


@gpu
@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("share", [0.5, 0.9, 0.95, 0.999])
@pytest.mark.parametrize("w", WINDOWS)
@pytest.mark.parametrize("context", [8192, 32768, 131072])
def test_sink_and_long_tail(lib, context, w, share, flat):
    top = Sink(context, share, w, 128, 4, flat).check()
    assert 0.2 < float(top.mean()) < 0.9999


@gpu
@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("w", WINDOWS)
@pytest.mark.parametrize("at", [700, 100001, (0, 130), (0, 1, 2, 3), (5, 3000)])
def test_sinks_elsewhere_and_several(lib, at, w, flat):
    Sink(131072, 0.95, w, 128, 4, flat, at=at).check()


@gpu
@pytest.mark.parametrize("share", [0.5, 0.9])
@pytest.mark.parametrize("w", WINDOWS)
@pytest.mark.parametrize("at", [0, 1000])
def test_sink_in_64_wide_heads(lib, at, w, share):
    Sink(20000, share, w, 64, 4, True, at=at, page=16).check()
    Sink(20000, share, w, 64, 4, False, at=at, page=128).check()


@gpu
@pytest.mark.parametrize("context", [60, 127, 300, 2000])
@pytest.mark.parametrize("w", WINDOWS)
def test_sink_over_short_contexts(lib, w, context):
    """The tail shares the dominant token's tile."""
    for share in (0.9, 0.95, 0.99, 0.999):
        for flat in (True, False):
            Sink(context, share, w, 128, 4, flat, page=32).check()
