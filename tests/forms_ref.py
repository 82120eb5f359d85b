"""64-bit attention over the cache's codes for any rule of what a row sees, and the bounds that the
tests of dspark_attend_sinks and dspark_attend_shared hold results to."""
import numpy as np
import torch

import cache_ref as ref


def attend(case, q, scale, seen):
    """q [rows, q_heads, dim] float64; seen(b, pos) -> token numbers. Returns out, lse and, for the
    tolerances, sum p |v| / l, the largest scale * sum |q k|, and what the softmax weights' pieces may
    be off by (2^-8 of a weight or 2^-16 of the largest, no more than the weight itself)."""
    rows, hq, D = q.shape
    n, heads, page = case.n, case.heads, case.page
    group = hq // heads
    out, lse = np.zeros((rows, hq, D)), np.full((rows, hq), -np.inf)
    spread, big, pieces = np.zeros((rows, hq, D)), np.zeros((rows, hq)), np.zeros((rows, hq, D))
    for b in range(len(case.lengths)):
        for r in range(case.cu[b], case.cu[b + 1]):
            t = np.asarray(seen(b, int(case.lengths[b]) + r - case.cu[b]), np.int64)
            j = t // page
            width = case.table.shape[1]
            ids = np.where(j < width, case.table[b, np.minimum(j, width - 1)], -1)
            ok = (ids >= 0) & (ids < n)
            t, ids = t[ok], ids[ok]
            if len(t) == 0:
                continue
            for h in range(heads):
                vs = case.scale["v"][ids, h].astype(np.float64)
                kk = ref.decode(case.codes["k"][ids, h, t % page]) * case.scale["k"][ids, h].astype(np.float64)[:, None]
                vv = ref.decode(case.codes["v"][ids, h, t % page]) * vs[:, None]
                g = slice(h * group, (h + 1) * group)
                s = scale * (q[r, g] @ kk.T)
                m = s.max(1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(1, keepdims=True)
                out[r, g], spread[r, g] = p @ vv / l, p @ np.abs(vv) / l
                w = p * vs[None, :]
                off = np.minimum(w, np.maximum(2.0 ** -8 * w, 2.0 ** -16 * w.max(1, keepdims=True)))
                pieces[r, g] = (off / vs[None, :]) @ np.abs(vv) / l
                lse[r, g] = (m + np.log(l))[:, 0]
                big[r, g] = abs(scale) * (np.abs(q[r, g]) @ np.abs(kk).T).max(1)
    return out, lse, spread, big, pieces


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
