"""Operators of a decode step's target forward, as measured: rotary positions, the append of a
step's keys and values to a paged 8-bit cache, and the ragged attention over that cache.

Every case is a dict of plain values; `prepare` makes its inputs from a seed, `run` makes one
pass, in plain torch (own = False) or through the library's calls (own = True), `exact` gives
the same outputs from the definitions in 64 bits.

Shapes. A step holds B requests; request b has w_b window rows (the anchor and its drafts, or a
piece of a prompt) packed one after another, and `lengths[b]` tokens in the cache before them.
Keys and values are e4m3 codes in pages [n_pages, kv_heads, page, dim] with one fp32 scale per
(page, head); `table[b, j]` is the page of request b's tokens j*page .. (j+1)*page - 1.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
WORKSPACE_BYTES = 64 << 20     # the caller's scratch for the attention
PAD = 8                        # packed rows are padded to a multiple of this (a capture tier)


# ---- cases -------------------------------------------------------------------------------
def _rotate(rows, heads, dim, rot, layout, dtype, inverse=False, far=131072, scaling="none"):
    return dict(op="rotate", rows=rows, heads=heads, dim=dim, rot=rot, layout=layout, dtype=dtype,
                inverse=inverse, far=far, scaling=scaling)


def _step(op, B, w, ctx, q_heads, kv_heads, dim, page, **more):
    return dict(op=op, B=B, w_lo=w[0], w_hi=w[1], ctx_lo=ctx[0], ctx_hi=ctx[1], q_heads=q_heads,
                kv_heads=kv_heads, dim=dim, page=page, **more)


def listed():
    half = dict(rot=128, layout="half", dtype="bf16", scaling="none")
    return [
        # queries and keys of one request's 16-row verify window
        dict(_rotate(16, 40, 128, 128, "half", "bf16"), name="rotate_one_window"),
        # a prompt's queries and keys, positions far beyond the trained context
        dict(_rotate(8192, 40, 128, 128, "half", "bf16", scaling="by_parts"),
             name="rotate_prompt_far"),
        # the gradient's way back through a partial, interleaved rotation
        dict(_rotate(4999, 24, 96, 64, "interleaved", "f32", inverse=True, far=32768,
                     scaling="linear"), name="rotate_grad_partial"),
        # batch-1 decode: one 16-row window (the latency workload's block)
        dict(_step("append", 1, (16, 16), (1000, 1000), 32, 8, 128, 16, **half),
             name="append_one_window"),
        # a batch of 256 requests with scheduled windows of 1..8 rows, inside a page or across two
        dict(_step("append", 256, (1, 8), (200, 2000), 32, 8, 128, 32, **half),
             name="append_verify_batch"),
        # prompts of odd lengths written into fresh pages
        dict(_step("append", 3, (1001, 7003), (0, 0), 32, 8, 128, 64, rot=128, layout="half",
                   dtype="bf16", scaling="by_parts"), name="append_prompts"),
        # batch-1 decode over a short context: latency
        dict(_step("attend", 1, (4, 4), (1000, 1000), 32, 8, 128, 16, window=0),
             name="attend_one_short"),
        # batch-1 decode over a long context: one request's cache spread over the whole GPU
        dict(_step("attend", 1, (5, 5), (131072, 131072), 32, 8, 128, 64, window=0),
             name="attend_one_long"),
        # the verify step of 256 requests, windows of 1..8 rows, ragged contexts
        dict(_step("attend", 256, (1, 8), (128, 2048), 32, 8, 128, 32, window=0),
             name="attend_verify_batch"),
        # plain decode, one row per request, long ragged contexts
        dict(_step("attend", 192, (1, 1), (1024, 8192), 32, 8, 128, 64, window=0),
             name="attend_single_tokens"),
        # a prompt's piece against the cache that holds its beginning
        dict(_step("attend", 2, (2000, 2048), (4097, 8191), 32, 8, 128, 64, window=0),
             name="attend_prompt_piece"),
        # 64-wide heads, three queries per key head, a sliding window, lengths from almost none
        dict(_step("attend", 33, (1, 7), (3, 5000), 12, 4, 64, 16, window=1000),
             name="attend_sliding_odd"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["rotate", "append", "append", "attend", "attend", "attend"])
    scaling = rng.choice(["none", "linear", "by_parts"])
    layout = rng.choice(["half", "interleaved"])
    if op == "rotate":
        dim = rng.choice([64, 96, 128, 256])
        return _rotate(_log(rng, 1, 8192), rng.randint(1, 40), dim, rng.choice([dim, dim // 2]),
                       layout, rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.4,
                       rng.choice([4096, 131072, 1000000]), scaling)
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        more = dict(rot=rng.choice([dim, dim // 2]), layout=layout,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), scaling=scaling)
        if rng.random() < 0.3:      # prompts
            hi = _log(rng, 64, 6000)
            return _step(op, rng.randint(1, 3), (max(1, hi // 3), hi), (0, rng.randint(0, 500)),
                         q_heads, kv_heads, dim, page, **more)
        hi = rng.randint(1, 16)
        c = _log(rng, 8, 4000)
        return _step(op, _log(rng, 1, 256), (rng.randint(1, hi), hi), (rng.randint(0, c), c),
                     q_heads, kv_heads, dim, page, **more)
    q_heads = min(q_heads, 32)
    window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    if rng.random() < 0.25:         # prompts and their pieces
        hi = _log(rng, 64, 2048)
        c = rng.randint(0, 8000)
        return _step(op, rng.randint(1, 2), (max(1, hi // 2), hi), (c // 2, c), q_heads, kv_heads,
                     dim, page, window=window)
    if rng.random() < 0.3:          # few requests, long contexts
        hi = rng.randint(1, 16)
        c = _log(rng, 2000, 100000)
        return _step(op, rng.randint(1, 4), (rng.randint(1, hi), hi), (c // 3, c), q_heads,
                     kv_heads, dim, page, window=window)
    hi = rng.randint(1, 8)
    c = _log(rng, 16, 3000)
    return _step(op, _log(rng, 4, 256), (rng.randint(1, hi), hi), (rng.randint(0, c), c), q_heads,
                 kv_heads, dim, page, window=window)


def _spread(lo, hi, n, log):
    """n whole numbers from lo to hi, evenly spread (over their logarithm): the same for every
    seed, so that a case's work is known; the seed only orders them."""
    if n == 1:
        return [hi]
    a, b = (math.log(lo + 1), math.log(hi + 1)) if log else (lo, hi)
    at = [a + (b - a) * i / (n - 1) for i in range(n)]
    return [int(round(math.exp(x) - 1 if log else x)) for x in at]


def _sizes(case):
    w = _spread(case["w_lo"], case["w_hi"], case["B"], False)
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], case["B"], True)
    return w, ctx


def work(case):
    if case["op"] == "rotate":
        n = case["rows"] * case["heads"] * case["dim"]
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * e + 4 * case["rows"],
                "flops": 3 * case["rows"] * case["heads"] * case["rot"]}
    w, ctx = _sizes(case)
    M, B = sum(w), case["B"]
    hq, hk, D, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "append":
        e = 2 if case["dtype"] == "bf16" else 4
        blocks = sum(-(-x // page) + 1 for x in w)
        return {"bytes": M * D * (2 * hq * e + 2 * hk * e + 2 * hk) + 8 * blocks * hk + 12 * M,
                "flops": M * D * (3 * hq + 6 * hk)}
    # tokens read and (row, token) pairs computed; windows and contexts meet in the seed's order,
    # so the pairs are the mean over the orders
    cap = case["window"] or 1 << 60
    mean_w = M / B
    tokens = sum(min(c + mean_w, cap + mean_w - 1) for c in ctx)
    pairs = M * sum(min(c + (mean_w + 1) / 2, cap) for c in ctx) / B
    return {"bytes": tokens * hk * (2 * D + 8 / page) + 4 * M * hq * D + 4 * M * hq,
            "flops": 4 * D * hq * pairs}


# ---- inputs ------------------------------------------------------------------------------
def _frequencies(rot, scaling, base=500000.0):
    """Radians per position of each rotated pair, and the factor on cos and sin: as trained, all
    positions divided (linear), or the slow pairs divided and the fast ones kept (by_parts)."""
    freq = [base ** (-2.0 * j / rot) for j in range(rot // 2)]
    if scaling == "linear":
        return [f / 4.0 for f in freq], 1.0
    if scaling == "by_parts":
        factor, trained, slow, fast = 16.0, 8192.0, 1.0, 32.0
        out = []
        for f in freq:
            keep = min(1.0, max(0.0, (trained * f / (2 * math.pi) - slow) / (fast - slow)))
            out.append((1 - keep) * f / factor + keep * f)
        return out, 0.1 * math.log(factor) + 1.0
    return freq, 1.0


def _rope_inputs(case, dev):
    freq, mscale = _frequencies(case["rot"], case["scaling"])
    turns = [int(f / (2 * math.pi) * 2.0 ** 64) for f in freq]
    turns = [t - (1 << 64) if t >= 1 << 63 else t for t in turns]
    return {"freq": torch.tensor(freq, dtype=torch.float64, device=dev), "mscale": mscale,
            "turns": torch.tensor(turns, dtype=torch.int64, device=dev)}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    s = {"case": case}
    if case["op"] == "rotate":
        # the rotated heads are the front of a projection's output row
        rows, heads, dim = case["rows"], case["heads"], case["dim"]
        s.update(_rope_inputs(case, dev))
        proj = torch.randn(rows, heads + 2, dim, generator=g, device=dev).to(dt)
        s["x"] = proj[:, :heads]
        s["positions"] = torch.randint(0, case["far"], (rows,), generator=g, device=dev,
                                       dtype=torch.int32)
        s["y"] = torch.zeros(rows, heads, dim, dtype=dt, device=dev)
        return s

    B, page, D = case["B"], case["page"], case["dim"]
    hq, hk = case["q_heads"], case["kv_heads"]
    w, ctx = _sizes(case)
    w = [w[i] for i in torch.randperm(B, generator=host).tolist()]
    ctx = [ctx[i] for i in torch.randperm(B, generator=host).tolist()]
    blocks = [-(-(c + n) // page) for c, n in zip(ctx, w)]
    most = [-(-(c + case["w_hi"]) // page) for c in ctx]      # whatever windows meet them
    n_pages = sum(most) + 3
    order = torch.randperm(n_pages, generator=host).tolist()
    table = torch.zeros(B, max(most), dtype=torch.int32)
    k = 0
    for b, n in enumerate(blocks):
        table[b, :n] = torch.tensor(order[k:k + n], dtype=torch.int32)
        k += n
    M = sum(w)
    rows = -(-M // PAD) * PAD
    cu = [0]
    for n in w:
        cu.append(cu[-1] + n)
    i32 = dict(dtype=torch.int32, device=dev)
    s.update(M=M, rows=rows, table=table.to(dev), lengths=torch.tensor(ctx, **i32),
             cu_seqlens=torch.tensor(cu, **i32), status=torch.zeros(1, **i32))
    # the cache as earlier steps left it: blocks of differing magnitude, scales a power of two
    # that keeps each block within e4m3's range
    for name in ("k", "v"):
        x = torch.randn(n_pages, hk, page, D, generator=g, device=dev)
        x *= torch.exp2(torch.rand(n_pages, hk, 1, 1, generator=g, device=dev) * 2 - 1)
        scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(2, 3)) / 448.0)))
        s[name + "_scale"] = scale
        s[name] = (x / scale[:, :, None, None]).to(FP8)
        del x
    proj = torch.randn(rows, (hq + 2 * hk), D, generator=g, device=dev).to(dt)
    if case["op"] == "append":
        s.update(_rope_inputs(case, dev))
        s.update(q=proj[:, :hq], new_k=proj[:, hq:hq + hk], new_v=proj[:, hq + hk:])
        req = torch.repeat_interleave(torch.arange(B), torch.tensor(w)).to(torch.int32)
        at = torch.cat([torch.arange(n) for n in w]).to(torch.int32)
        pad = torch.full((rows - M,), -1, dtype=torch.int32)
        s["row_req"] = torch.cat([req, pad]).to(dev)
        s["row_pos"] = torch.cat([at, pad]).to(dev)
        s["q_out"] = torch.zeros(rows, hq, D, dtype=dt, device=dev)
        return s
    s["q"] = proj[:, :hq].contiguous()
    # a stale slot may hold anything: the slots after each request's last token are NaN codes
    for b in range(min(B, 4)):
        used = (ctx[b] + w[b]) - (blocks[b] - 1) * page
        last = int(table[b, blocks[b] - 1])
        s["k"].view(torch.uint8)[last, :, used:] = 0x7F
        s["v"].view(torch.uint8)[last, :, used:] = 0x7F
    s["out"] = torch.zeros(rows, hq, D, dtype=dt, device=dev)
    s["lse"] = torch.zeros(rows, hq, dtype=torch.float32, device=dev)
    s["workspace"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
    return s


# ---- the plain forms ---------------------------------------------------------------------
def _turn(x, positions, freq, mscale, rot, layout, inverse=False):
    """x [rows, heads, dim] fp32, rotated; angles in 64 bits, products in 32."""
    angle = positions.double()[:, None] * freq
    c = (torch.cos(angle) * mscale).float()[:, None]
    s = (torch.sin(angle) * (-mscale if inverse else mscale)).float()[:, None]
    y = x.clone()
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    return y


def _plain_rotate(s):
    c = s["case"]
    return _turn(s["x"].float(), s["positions"], s["freq"], s["mscale"], c["rot"], c["layout"],
                 c["inverse"]).to(s["x"].dtype)


def _power_scale(amax):
    """The smallest power of two 2^e, e >= -64, with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.ldexp(torch.ones_like(amax), torch.clamp(e, min=-64))


def _plain_append_one(pages, scale, rows, ids, slot):
    """Appends rows [M, heads, dim] (fp32) to `pages` at (ids, slot), in place."""
    touched, at = torch.unique(ids, return_inverse=True)
    T, hk, page = touched.numel(), pages.shape[1], pages.shape[2]
    amax = torch.zeros(T, hk, device=rows.device).index_reduce_(0, at, rows.abs().amax(-1), "amax")
    first = torch.full((T,), page, device=rows.device).scatter_reduce_(0, at, slot, "amin")
    old, new = scale[touched], _power_scale(amax)
    new = torch.where((first > 0)[:, None], torch.maximum(old, new), new)
    codes = pages.view(torch.uint8)
    tile = codes[touched]
    again = (tile.view(FP8).float() * (old / new)[:, :, None, None]).to(FP8).view(torch.uint8)
    kept = torch.arange(page, device=rows.device)[None, :] < first[:, None]
    tile = torch.where(kept[:, None, :, None], again, tile)
    tile[at, :, slot] = (rows / new[at][:, :, None]).to(FP8).view(torch.uint8)
    codes[touched] = tile
    scale[touched] = new


def _plain_append(s):
    c, M = s["case"], s["M"]
    req, i = s["row_req"][:M].long(), s["row_pos"][:M].long()
    pos = s["lengths"].long()[req] + i
    ids, slot = s["table"].long()[req, pos // c["page"]], pos % c["page"]
    turn = (pos, s["freq"], s["mscale"], c["rot"], c["layout"])
    s["q_out"][:M] = _turn(s["q"][:M].float(), *turn).to(s["q"].dtype)
    _plain_append_one(s["k"], s["k_scale"], _turn(s["new_k"][:M].float(), *turn), ids, slot)
    _plain_append_one(s["v"], s["v_scale"], s["new_v"][:M].float(), ids, slot)
    return s["q_out"], s["k"], s["v"], s["k_scale"], s["v_scale"]


def _plain_attend(s):
    c, M = s["case"], s["M"]
    B, D, page, hk = c["B"], c["dim"], c["page"], c["kv_heads"]
    group = c["q_heads"] // hk
    dev = s["q"].device
    w = (s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]).long()
    W, L = c["w_hi"], s["table"].shape[1] * page
    # queries [B, hk, W * group, D], rows past a request's window repeat its last
    i = torch.minimum(torch.arange(W, device=dev)[None, :], w[:, None] - 1)
    row = s["cu_seqlens"][:-1].long()[:, None] + i
    q = s["q"][row].float().view(B, W, hk, group, D).permute(0, 2, 1, 3, 4)
    q = q.reshape(B, hk, W * group, D)
    t = torch.arange(L, device=dev)
    total = s["lengths"].long() + w
    here = t[None, :] < total[:, None]                                     # [B, L]

    def gather(name):
        ids = s["table"].long()
        x = s[name].view(torch.uint8)[ids].view(FP8).float()               # [B, n, hk, page, D]
        x *= s[name + "_scale"][ids][:, :, :, None, None]
        x = x.permute(0, 2, 1, 3, 4).reshape(B, hk, L, D)
        return x.masked_fill_(~here[:, None, :, None], 0.0)

    score = torch.matmul(q, gather("k").transpose(2, 3)) * (1.0 / math.sqrt(D))
    pos = s["lengths"].long()[:, None] + i                                 # [B, W]
    seen = t[None, None, :] <= pos[:, :, None]
    if c["window"]:
        seen &= t[None, None, :] > pos[:, :, None] - c["window"]
    seen = seen[:, None, :, None, :].expand(B, hk, W, group, L).reshape(B, hk, W * group, L)
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score, gather("v")) / total
    lse = (torch.log(total) + top)[..., 0]
    out = out.view(B, hk, W, group, D).permute(0, 2, 1, 3, 4).reshape(B, W, hk * group, D)
    lse = lse.view(B, hk, W, group).permute(0, 2, 1, 3).reshape(B, W, hk * group)
    take = torch.arange(W, device=dev)[None, :] < w[:, None]
    s["out"][:M] = out[take].to(s["out"].dtype)
    s["lse"][:M] = lse[take]
    return s["out"], s["lse"]


def run(s):
    if not own:
        return {"rotate": _plain_rotate, "append": _plain_append, "attend": _plain_attend}[
            s["case"]["op"]](s)
    if "call" not in s:
        s["call"], s["result"] = _call(s)      # checked and marshalled once for these buffers
    s["call"]()
    return s["result"]


def _call(s):
    """The library's prepared call on a state's buffers, as a decode loop keeps it."""
    from speculative_decoding_ragged_gb300 import _binding as bd
    c = s["case"]
    if c["op"] != "attend":
        rope = bd.Rope(s["turns"], s["mscale"], interleaved=c["layout"] == "interleaved")
    if c["op"] == "rotate":
        call = bd.dspark_rotate(s["x"], s["y"], s["positions"], rope, inverse=c["inverse"],
                                prepare=True)
        return call, s["y"]
    cache = bd.PagedCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"])
    if c["op"] == "append":
        call = bd.dspark_append(cache, s["new_k"], s["new_v"], s["row_req"], s["row_pos"],
                                s["lengths"], rope=rope, q=s["q"], q_out=s["q_out"],
                                status=s["status"], prepare=True)
        return call, (s["q_out"], s["k"], s["v"], s["k_scale"], s["v_scale"])
    call = bd.dspark_attend(cache, s["q"], s["out"], s["cu_seqlens"], s["lengths"],
                            s["workspace"], window=c["window"], lse=s["lse"],
                            status=s["status"], prepare=True)
    return call, (s["out"], s["lse"])


# ---- 64 bits -----------------------------------------------------------------------------
def _exact_turn(x, positions, case, inverse):
    """Each pair as a complex number times mscale * exp(+-i * position * frequency)."""
    freq, mscale = _frequencies(case["rot"], case["scaling"])
    x, rot = x.double(), case["rot"]
    angle = torch.outer(positions.double(), torch.tensor(freq, dtype=torch.float64,
                                                         device=x.device))
    factor = torch.polar(torch.full_like(angle, mscale), -angle if inverse else angle)[:, None]
    head, tail = x[..., :rot], x[..., rot:]
    if case["layout"] == "half":
        z = torch.complex(head[..., :rot // 2], head[..., rot // 2:]) * factor
        return torch.cat([z.real, z.imag, tail], -1)
    z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * factor
    return torch.cat([torch.view_as_real(z).flatten(-2), tail], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_turn(s["x"], s["positions"], case, case["inverse"])
    cu, lengths = s["cu_seqlens"].tolist(), s["lengths"].tolist()
    table, page, B = s["table"].tolist(), case["page"], case["B"]
    if case["op"] == "append":
        q_out = s["q_out"].double()
        out = {n: s[n].double() for n in ("k", "v", "k_scale", "v_scale")}
        for b in range(B):
            rows = slice(cu[b], cu[b + 1])
            pos = torch.arange(lengths[b], lengths[b] + cu[b + 1] - cu[b], device=q_out.device)
            q_out[rows] = _exact_turn(s["q"][rows], pos, case, False)
            new = {"k": _exact_turn(s["new_k"][rows], pos, case, False),
                   "v": s["new_v"][rows].double()}
            at = lengths[b]
            while at < lengths[b] + cu[b + 1] - cu[b]:
                slot, p = at % page, table[b][at // page]
                n = min(page - slot, lengths[b] + cu[b + 1] - cu[b] - at)
                for name in ("k", "v"):
                    x = new[name][at - lengths[b]:at - lengths[b] + n].transpose(0, 1)
                    top = x.abs().amax(dim=(1, 2))
                    e = torch.ceil(torch.log2(top / 448.0)).clamp(min=-64)
                    scale = torch.exp2(e)
                    if slot:
                        old = out[name + "_scale"][p]
                        scale = torch.maximum(scale, old)
                        kept = out[name][p, :, :slot] * (old / scale)[:, None, None]
                        out[name][p, :, :slot] = kept.to(FP8).double()
                    # 32 bits hold a value's e4m3 neighbours and their midpoint exactly
                    codes = (x / scale[:, None, None]).float().to(FP8)
                    out[name][p, :, slot:slot + n] = codes.double()
                    out[name + "_scale"][p] = scale
                at += n
        return q_out, out["k"], out["v"], out["k_scale"], out["v_scale"]
    if work(case)["flops"] > 3e12:      # FP64 is slow on this part
        return None
    D, hk = case["dim"], case["kv_heads"]
    group = case["q_heads"] // hk
    out, lse = s["out"].double(), s["lse"].double()
    for b in range(B):
        n, w = lengths[b] + cu[b + 1] - cu[b], cu[b + 1] - cu[b]
        ids = s["table"][b, :-(-n // page)].long()

        def cached(name):
            x = s[name].view(torch.uint8)[ids].view(FP8).double()
            x = x * s[name + "_scale"][ids].double()[:, :, None, None]
            return x.transpose(0, 1).reshape(hk, -1, D)[:, :n]

        k, v = cached("k"), cached("v")
        q = s["q"][cu[b]:cu[b + 1]].double().view(w, hk, group, D)
        t = torch.arange(n, device=q.device)[None, :]
        pos = torch.arange(lengths[b], n, device=q.device)[:, None]
        hide = t > pos
        if case["window"]:
            hide = hide | (t <= pos - case["window"])
        score = torch.einsum("whgd,htd->hgwt", q, k) / math.sqrt(D)
        score = score.masked_fill(hide, -math.inf)
        lse[cu[b]:cu[b + 1]] = torch.logsumexp(score, -1).permute(2, 0, 1).reshape(w, -1)
        p = torch.softmax(score, -1)
        out[cu[b]:cu[b + 1]] = torch.einsum("hgwt,htd->whgd", p, v).reshape(w, -1, D)
    return out, lse
