"""64-bit attention over the cache's codes for any rule of what a row sees, and the bounds that the
tests of dspark_attend_sinks and dspark_attend_shared hold results to."""
import numpy as np
import torch


def attend(case, q, scale, seen):
    """q [rows, q_heads, dim] float64; seen(b, pos) -> token numbers. Returns out, lse and, for the
    tolerances, sum p |v| / l, the largest scale * sum |q k|, and what the softmax weights' pieces may
    be off by (2^-8 of a weight or 2^-16 of the largest, no more than the weight itself). Request by
    request, on the GPU's 64-bit units."""
    dev = torch.device("cuda:0")
    put = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(dev)       # noqa: E731
    rows, hq, D = q.shape
    n, heads, page = case.n, case.heads, case.page
    group = hq // heads
    K, V = (put(case.codes[x]).view(torch.float8_e4m3fn).double() * put(case.scale[x]).double()[:, :, None, None]
            for x in "kv")
    scale_v, table, q = put(case.scale["v"]).double(), put(case.table).long(), put(q).double()
    f64 = dict(dtype=torch.float64, device=dev)
    out, lse = torch.zeros(rows, hq, D, **f64), torch.full((rows, hq), -np.inf, **f64)
    spread, big, pieces = torch.zeros_like(out), torch.zeros(rows, hq, **f64), torch.zeros_like(out)
    for b in range(len(case.lengths)):
        r0, r1 = int(case.cu[b]), int(case.cu[b + 1])
        if r1 <= r0:
            continue
        tokens = [np.asarray(seen(b, int(case.lengths[b]) + i), np.int64) for i in range(r1 - r0)]
        t = np.unique(np.concatenate(tokens))
        hide = put(np.stack([~np.isin(t, x) for x in tokens]))
        t = put(t)
        j = t // page
        ids = torch.where(j < table.shape[1], table[b, j.clamp(max=table.shape[1] - 1)], -1)
        there = (ids >= 0) & (ids < n)
        ids = ids.clamp(0, n - 1)
        hide = (hide | ~there)[None, None]                                 # [1, 1, w, T]
        k, v = (x[ids, :, t % page].transpose(0, 1) for x in (K, V))       # [heads, T, D]
        k, v = k.masked_fill(~there[None, :, None], 0.0), v.masked_fill(~there[None, :, None], 0.0)
        vs = scale_v[ids].T[:, None, None]                                 # [heads, 1, 1, T]
        x = q[r0:r1].view(r1 - r0, heads, group, D).permute(1, 2, 0, 3)    # [heads, group, w, D]
        s = (scale * (x @ k[:, None].mT)).masked_fill(hide, -np.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(torch.isinf(m), 0.0, m))
        l = p.sum(-1, keepdim=True)
        some = l > 0
        w = p * vs
        off = torch.minimum(w, torch.maximum(2.0 ** -8 * w, 2.0 ** -16 * w.amax(-1, keepdim=True))) / vs
        over = torch.where(some, l, 1.0)
        back = lambda y: y.permute(2, 0, 1, 3).reshape(r1 - r0, hq, -1)     # noqa: E731
        out[r0:r1] = back(p @ v[:, None] / over)
        spread[r0:r1] = back(p @ v[:, None].abs() / over)
        pieces[r0:r1] = back(off @ v[:, None].abs() / over)
        lse[r0:r1] = back(torch.where(some, m + torch.log(over), -np.inf))[..., 0]
        sums = (x.abs() @ k[:, None].abs().mT * abs(scale)).masked_fill(hide, 0.0)
        big[r0:r1] = back(sums.amax(-1, keepdim=True))[..., 0]
    return tuple(y.cpu().numpy() for y in (out, lse, spread, big, pieces))


def check(case, dtype, q, out, lse, seen, *, joined=False, scale=None):
    """A call's results (float64, sentinel 5.0 in the rows behind the packed ones) against attend.

    A score: dim products and sums in fp32 and the factors' roundings; on the tensor cores q's pieces
    too, 2^-17 of the row's largest. exp2, the order of sums and the division: 2^-20 together. Joined
    parts (a prefix's and the own tokens'): each one's log2 sum is rounded to fp32, 2^-24 of its
    magnitude, which the weights take as ln 2 of that, twice, and the shares' own few roundings."""
    dim, M = case.dim, int(case.cu[-1])
    a = dim ** -0.5 if scale is None else scale
    want, wl, spread, big, pieces = (x[:M] for x in attend(case, q, a, seen))
    assert (out[M:] == 5.0).all()
    fast = dtype == torch.bfloat16 and dim in (64, 128)
    ds = (dim + 8) * 2.0 ** -24 * big
    if fast:
        ds = ds + 2.0 ** -17 * dim * abs(a) * np.abs(q[:M]).max(-1) * (448.0 * case.scale["k"]).max()
    empty = np.isneginf(wl)
    size = np.abs(np.where(empty, 0, wl))
    join = 2.0 ** -22 * (2 + size) if joined else 0.0
    tol = spread * (np.exp(2 * ds) - 1 + 2.0 ** -20 + join)[..., None]
    if fast:
        tol = tol + pieces
    tol = tol + torch.finfo(dtype).eps / 2 * (np.abs(want) + tol) + 1e-30
    err = np.abs(out[:M] - want)
    assert (err <= tol).all(), (float(err.max()), float((err - tol).max()))
    assert (out[:M][empty] == 0).all()
    if lse is not None:
        assert (np.isneginf(lse[:M]) == empty).all()
        e = np.abs(np.where(empty, 0, lse[:M]) - np.where(empty, 0, wl))
        assert (e <= 2 * ds + 2.0 ** -20 * (1 + size) + join).all(), e.max()
        assert (lse[M:] == 5.0).all()
