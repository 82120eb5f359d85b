"""Plain 64-bit implementations of the target forward's ragged operators (numpy, on the host),
written from include/dspark.h: rotary positions, the append to the paged 8-bit cache, the
attention over it. The tests of those operators compare the library with these."""
from __future__ import annotations

import numpy as np

# every finite e4m3 magnitude, in order: code c (0..126) stands for E4M3[c]
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def decode(codes):
    """uint8 e4m3 codes -> float64 (0x7f, 0xff: NaN)."""
    codes = np.asarray(codes)
    mag = np.append(E4M3, np.nan)[codes & 0x7f]
    return np.where(codes & 0x80, -mag, mag)


def encode(x):
    """float64 -> e4m3 codes, nearest, ties to the even code, saturating at 448."""
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(E4M3, a), 1, 126)
    lo = hi - 1
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def half_step(y):
    """Half the distance between e4m3's neighbours at |y| (in units of the scale)."""
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    return 2.0 ** (e - 4)


def rotate(x, positions, turns, mscale, interleaved, inverse=False):
    """x [rows, heads, dim] float64; the angle is exact: an integer product modulo 2^64."""
    half = len(turns)
    y = np.array(x, dtype=np.float64)
    if half == 0:
        return y
    phase = np.array([[(int(p) * int(t)) % (1 << 64) / 2.0 ** 64 for t in turns]
                      for p in positions]).reshape(len(positions), half)
    c = mscale * np.cos(2 * np.pi * phase)[:, None]
    s = mscale * np.sin(2 * np.pi * phase)[:, None] * (-1 if inverse else 1)
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    return y


# |computed - exact| of a rotated element over mscale (|a| + |b|): the angle's conversion to fp32
# (2^-25 half turns: 9.4e-8 rad), cos and sin (2 ulp: 2.4e-7), the factor mscale, two products
# and their sum (3 * 2^-24 * 2: 3.6e-7)
ROTATE_TOL = 7e-7


def rotate_bound(x, half, mscale, interleaved):
    """ROTATE_TOL's |a| + |b| of every element (0 past the rotated part)."""
    z = np.zeros(x.shape)
    if half:
        if interleaved:
            t = np.abs(x[..., 0:2 * half:2]) + np.abs(x[..., 1:2 * half:2])
            z[..., 0:2 * half:2] = z[..., 1:2 * half:2] = t
        else:
            t = np.abs(x[..., :half]) + np.abs(x[..., half:2 * half])
            z[..., :half] = z[..., half:2 * half] = t
    return z * abs(mscale) * ROTATE_TOL


def fresh_scale(amax):
    e = -64
    if amax > 0:
        e = max(-64, int(np.floor(np.log2(amax))) - 10)
        while 448.0 * 2.0 ** e < amax:
            e += 1
    return 2.0 ** e


def append(codes, scale, x, row_req, row_pos, lengths, table):
    """x [rows, heads, dim] (already rotated) into codes uint8 [n, heads, page, dim] and scale
    [n, heads], in place. Rows must be valid. Returns {(page, head): x's rows and first slot}."""
    page, heads = codes.shape[2], codes.shape[1]
    blocks = {}
    for r, (b, i) in enumerate(zip(row_req, row_pos)):
        if b < 0:
            continue
        t = int(lengths[b]) + int(i)
        blocks.setdefault(int(table[b, t // page]), []).append((t % page, r))
    for p, rows in blocks.items():
        slots, rr = [s for s, _ in rows], [r for _, r in rows]
        for h in range(heads):
            v = np.where(np.isfinite(x[rr, h]), x[rr, h], 0.0)
            s = fresh_scale(np.abs(v).max())
            first = min(slots)
            if first > 0:
                old = float(scale[p, h])
                s = max(s, old)
                codes[p, h, :first] = encode(decode(codes[p, h, :first]) * (old / s))
            codes[p, h, slots] = encode(v / s)
            scale[p, h] = s
    return blocks


def attend(q, k, v, k_scale, v_scale, table, lengths, cu, scale, window=0):
    """q [rows, q_heads, dim] float64; codes and scales as stored. Returns out, lse and, for the
    tolerances, sum_t p_t |v_t| / l, the largest scale * sum_d |q_d k_td| of each row, and what
    weights of two e4m3 pieces may be off by: a weight (with its value's scale) is off by 2^-8 of
    itself or 2^-16 of the row's largest, whichever is more, and by no more than itself."""
    rows, hq, D = q.shape
    n, heads, page, _ = k.shape
    group = hq // heads
    out, lse = np.zeros((rows, hq, D)), np.full((rows, hq), -np.inf)
    spread, big = np.zeros((rows, hq, D)), np.zeros((rows, hq))
    pieces = np.zeros((rows, hq, D))
    for b in range(len(lengths)):
        for r in range(cu[b], cu[b + 1]):
            pos = int(lengths[b]) + r - cu[b]
            lo = max(0, pos - window + 1) if window else 0
            t = np.arange(lo, pos + 1)
            j = t // page
            ids = np.where(j < table.shape[1], table[b, np.minimum(j, table.shape[1] - 1)], -1)
            ok = (ids >= 0) & (ids < n)
            t, ids = t[ok], ids[ok]
            if len(t) == 0:
                continue
            for h in range(heads):
                kk = decode(k[ids, h, t % page]) * k_scale[ids, h].astype(np.float64)[:, None]
                vv = decode(v[ids, h, t % page]) * v_scale[ids, h].astype(np.float64)[:, None]
                g = slice(h * group, (h + 1) * group)
                s = scale * (q[r, g] @ kk.T)
                m = s.max(1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(1, keepdims=True)
                out[r, g] = p @ vv / l
                spread[r, g] = p @ np.abs(vv) / l
                vs = v_scale[ids, h].astype(np.float64)[None, :]
                w = p * vs
                off = np.minimum(w, np.maximum(2.0 ** -8 * w, 2.0 ** -16 * w.max(1, keepdims=True)))
                pieces[r, g] = (off / vs) @ np.abs(vv) / l
                lse[r, g] = (m + np.log(l))[:, 0]
                big[r, g] = abs(scale) * (np.abs(q[r, g]) @ np.abs(kk).T).max(1)
    return out, lse, spread, big, pieces
