"""More operators of a decode step, as measured: the logits' adjustments before verify (penalties
for repeated tokens, biases, grammar masks), and two more forms of the ragged attention over the
paged 8-bit cache: a sliding window whose first tokens stay visible (sinks), and requests that
share a prefix, computed once for all of them.

Every case is a dict of plain values; `prepare` makes its inputs from a seed, `run` makes one
pass, in plain torch (own = False) or through the library's calls (own = True), `exact` gives
the same outputs from the definitions in 64 bits.

Shapes. A step holds B requests; request b has w_b window rows (the anchor and its drafts, or a
piece of a prompt) packed one after another. Attention: `lengths[b]` tokens lie in the cache before
them; keys and values are e4m3 codes in pages [n_pages, kv_heads, page, dim] with one fp32 scale
per (page, head); `table[b, j]` is the page of request b's tokens j*page .. (j+1)*page - 1. Logits:
one row of V per packed row; request b's tokens so far are history[b, :history_len[b]], of which
the first prompt_len[b] are its prompt, and the last is the block's anchor, block_tokens[b, 0].
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
WORKSPACE_BYTES = 64 << 20     # the caller's scratch for the attention with sinks
PAD = 8                        # packed rows are padded to a multiple of this (a capture tier)


# ---- cases -------------------------------------------------------------------------------
def _adjust(B, w, V, history, dtype, penalties, bias, masked):
    """history: tokens per request, from and to; bias: the most entries of a request; masked: the
    share of requests under a grammar."""
    return dict(op="adjust", B=B, w_lo=w[0], w_hi=w[1], V=V, hist_lo=history[0],
                hist_hi=history[1], dtype=dtype, penalties=penalties, bias=bias, masked=masked)


def _step(op, B, w, ctx, q_heads, kv_heads, dim, page, **more):
    return dict(op=op, B=B, w_lo=w[0], w_hi=w[1], ctx_lo=ctx[0], ctx_hi=ctx[1], q_heads=q_heads,
                kv_heads=kv_heads, dim=dim, page=page, **more)


def _shared(groups, each, w, prefix, ctx, q_heads, kv_heads, dim, page):
    """groups of `each` requests behind a prefix; ctx: a request's own tokens after it."""
    return _step("shared", groups * each, w, ctx, q_heads, kv_heads, dim, page, groups=groups,
                 prefix_lo=prefix[0], prefix_hi=prefix[1])


def listed():
    return [
        # batch-1 decode: one 8-row window of one request with a short chat behind it: latency
        dict(_adjust(1, (8, 8), 151936, (1000, 1000), "bf16", True, 20, 0.0),
             name="adjust_one_window"),
        # the verify step of 256 requests, all with penalties and some biases
        dict(_adjust(256, (1, 8), 151936, (64, 4096), "bf16", True, 300, 0.0),
             name="adjust_verify_batch"),
        # structured output: every row under its grammar, nothing else to adjust
        dict(_adjust(128, (1, 4), 151936, (0, 0), "bf16", False, 0, 1.0), name="adjust_grammar"),
        # a mixed batch over an odd vocabulary, fp32 logits, everything at once
        dict(_adjust(33, (1, 5), 32003, (0, 9000), "f32", True, 100, 0.5), name="adjust_mixed_odd"),
        # batch-1 decode far into a stream: a window of the last tokens and the first few
        dict(_step("sinks", 1, (5, 5), (131072, 131072), 32, 8, 128, 64, window=4096, sinks=4),
             name="sinks_one_far"),
        # the verify step of 256 requests, contexts inside and beyond the window
        dict(_step("sinks", 256, (1, 8), (128, 8192), 32, 8, 128, 32, window=1024, sinks=4),
             name="sinks_verify_batch"),
        # pieces of two prompts
        dict(_step("sinks", 2, (2000, 2048), (4097, 8191), 32, 8, 128, 64, window=2000, sinks=128),
             name="sinks_prompt_piece"),
        # 64-wide heads, three queries per key head, a short window, sinks past a page
        dict(_step("sinks", 33, (1, 7), (3, 5000), 12, 4, 64, 16, window=100, sinks=19),
             name="sinks_short_odd"),
        # four samples of one question: latency
        dict(_shared(1, 4, (4, 4), (1000, 1000), (20, 60), 32, 8, 128, 16),
             name="shared_few_short"),
        # plain decode of 192 requests behind one long system prompt
        dict(_shared(1, 192, (1, 1), (16384, 16384), (1, 1000), 32, 8, 128, 64),
             name="shared_single_tokens"),
        # the verify step of 256 requests behind one prompt with examples
        dict(_shared(1, 256, (1, 8), (8192, 8192), (16, 1024), 32, 8, 128, 32),
             name="shared_verify_batch"),
        # sampled answers: 12 questions of uneven lengths with 7 answers each, 64-wide heads
        dict(_shared(12, 7, (1, 6), (300, 5000), (1, 700), 12, 4, 64, 16),
             name="shared_answers_odd"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["adjust", "sinks", "shared"])
    if op == "adjust":
        V = rng.choice([_log(rng, 500, 151936), _log(rng, 8000, 151936), 151936])
        hi = rng.randint(1, 8)
        w = (rng.randint(1, hi), hi)
        h = _log(rng, 4, 9000)
        penalties = rng.random() < 0.75
        return _adjust(_log(rng, 1, min(256, 2304 // sum(w))), w, V, (rng.randint(0, h), h),
                       rng.choice(["bf16", "bf16", "f32"]) if V < 70000 else "bf16", penalties,
                       rng.choice([0, rng.randint(1, 300)]),
                       rng.choice([0.0, 0.3, 1.0]) if penalties else rng.choice([0.3, 1.0]))
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    q_heads = min(32, kv_heads * rng.choice([1, 2, 3, 4, 8]))
    page = rng.choice([16, 32, 64, 128])
    hi = rng.randint(1, 8)
    w = (rng.randint(1, hi), hi)
    most = min(256, 2304 // sum(w))         # requests
    if op == "sinks":
        window, sinks = _log(rng, 1, 4096), _log(rng, 1, 300)
        at = rng.random()
        if at < 0.25:               # prompts and their pieces
            hi = _log(rng, 64, 2048)
            c, window = rng.randint(0, 8000), min(window, 2048)
            return _step(op, rng.randint(1, 2), (max(1, hi // 2), hi), (c // 2, c), q_heads,
                         kv_heads, dim, page, window=window, sinks=sinks)
        if at < 0.5:                # few requests, long contexts
            c = _log(rng, 2000, 130000)
            return _step(op, rng.randint(1, 4), w, (c // 3, c), q_heads, kv_heads, dim, page,
                         window=window, sinks=sinks)
        c = _log(rng, 16, 8000)
        return _step(op, _log(rng, 4, most), w, (rng.randint(0, c), c), q_heads, kv_heads, dim,
                     page, window=min(window, 1024), sinks=sinks)
    groups = rng.choice([1, 1, _log(rng, 2, 16)])
    each = _log(rng, 2, most // groups)
    p = _log(rng, 40, 8192)
    c = _log(rng, 2, 1000)
    return _shared(groups, each, w, (rng.randint(p // 3, p), p), (rng.randint(0, c), c), q_heads,
                   kv_heads, dim, page)


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


def _prefixes(case):
    """The groups' shared tokens: whole pages."""
    p = _spread(case["prefix_lo"], case["prefix_hi"], case["groups"], True)
    return [n // case["page"] * case["page"] for n in p]


def work(case):
    w = _spread(case["w_lo"], case["w_hi"], case["B"], False)
    M, B = sum(w), case["B"]
    if case["op"] == "adjust":
        e, V = 2 if case["dtype"] == "bf16" else 4, case["V"]
        tokens = sum(_spread(case["hist_lo"], case["hist_hi"], B, True)) if case["penalties"] else 0
        return {"bytes": 2 * e * M * V + case["masked"] * M * V / 8 + 4 * tokens +
                8 * B * case["bias"] / 2, "flops": 4 * M * V}
    _, ctx = _sizes(case)
    hq, hk, D, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    # tokens read and (row, token) pairs computed; windows and contexts meet in the seed's order,
    # so the pairs are the mean over the orders
    mean_w = M / B
    if case["op"] == "sinks":
        cap, sinks = case["window"], case["sinks"]
        tokens = sum(min(c + mean_w, cap + mean_w - 1 + sinks) for c in ctx)
        pairs = M * sum(min(c + (mean_w + 1) / 2, cap + sinks) for c in ctx) / B
    else:
        p = _prefixes(case)
        tokens = sum(p) + sum(ctx) + M
        pairs = M * (sum(p) / len(p) + sum(ctx) / B + (mean_w + 1) / 2)
    return {"bytes": tokens * hk * (2 * D + 8 / page) + 4 * M * hq * D + 4 * M * hq,
            "flops": 4 * D * hq * pairs}


# ---- inputs ------------------------------------------------------------------------------
def _generators(seed):
    dev = torch.device("cuda")
    g, host = torch.Generator(device=dev), torch.Generator()
    g.manual_seed(seed)
    host.manual_seed(seed)
    return dev, g, host


def _packed(w, rows, dev):
    """cu_seqlens, and the packed rows' requests and positions (padding: -1)."""
    B, M = len(w), sum(w)
    n = torch.tensor(w)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
    req = torch.repeat_interleave(torch.arange(B), n)
    at = torch.arange(M) - cu[req]
    pad = torch.full((rows - M,), -1)
    return [t.to(torch.int32).to(dev) for t in (cu, torch.cat([req, pad]), torch.cat([at, pad]))]


def _prepare_adjust(case, seed):
    dev, g, host = _generators(seed)
    B, V = case["B"], case["V"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    w = _spread(case["w_lo"], case["w_hi"], B, False)
    w = [w[i] for i in torch.randperm(B, generator=host).tolist()]
    M = sum(w)
    rows = -(-M // PAD) * PAD
    cu, row_req, row_pos = _packed(w, rows, dev)
    s = dict(case=case, M=M, cu_seqlens=cu, row_req=row_req, row_pos=row_pos,
             status=torch.zeros(1, dtype=torch.int32, device=dev))
    s["logits"] = (torch.randn(rows, V, generator=g, device=dev) * 2.5).to(dt)
    s["out"] = torch.zeros(rows, V, dtype=dt, device=dev)
    gamma = case["w_hi"]

    def tokens(*shape):             # some tokens come again and again
        return (V * torch.rand(*shape, generator=g, device=dev) ** 4).to(torch.int32).clamp_(0, V - 1)

    s["block_tokens"] = tokens(B, gamma)
    more = {}
    if case["penalties"]:
        n = _spread(case["hist_lo"], case["hist_hi"], B, True)
        n = torch.tensor([n[i] for i in torch.randperm(B, generator=host).tolist()])
        cap = max(1, int(n.max()) + 16)                 # the histories' buffer has room to grow
        history = tokens(B, cap)
        history.masked_fill_(torch.arange(cap, device=dev) >= n.to(dev)[:, None], -1)
        at = torch.rand(3, B, generator=host)
        more.update(history=history, history_len=n.to(torch.int32).to(dev),
                    prompt_len=(n * at[0]).to(torch.int32).to(dev),
                    repetition=(1.0 + 0.3 * at[1]).to(dev), presence=(at[2] * 0.8).to(dev),
                    frequency=((1 - at[2]) * 0.4).to(dev))
    if case["bias"]:
        # distinct tokens per request: a stretch of the vocabulary with a stride
        n = torch.randint(0, case["bias"] + 1, (B,), generator=host)
        step = max(1, V // (case["bias"] + 1))
        first = torch.randint(0, V, (B, 1), generator=host)
        ids = (first + step * torch.arange(case["bias"])) % V
        values = torch.randn(B, case["bias"], generator=host) * 4.0
        values[:, ::7] = -math.inf                      # a banned token
        more.update(bias_tokens=ids.to(torch.int32).to(dev), bias_values=values.to(dev),
                    bias_len=n.to(torch.int32).to(dev))
    if case["masked"]:
        # grammars: within a structure a few tokens are allowed, inside a string nearly all
        words = -(-V // 32)
        wide = torch.rand(rows, 1, generator=g, device=dev) < 0.3
        mask = torch.where(wide, -1, 0).to(torch.int32).expand(rows, words).clone()
        n = min(40, words)                              # in words of their own
        some = torch.randint(0, words, (rows, 1), generator=g, device=dev)
        some = (some + words // n * torch.arange(n, device=dev)) % words
        bit = torch.randint(0, 32, (rows, n), generator=g, device=dev)
        bit = (torch.ones_like(bit) << bit).to(torch.int32)
        mask.scatter_(1, some, torch.where(wide, ~bit, bit))
        who = torch.rand(B, generator=g, device=dev) < case["masked"]
        mine = who[row_req.clamp(min=0).long()] & (row_req >= 0)
        more["mask"] = mask
        more["mask_row"] = torch.where(mine, torch.arange(rows, device=dev), -1).to(torch.int32)
    s["more"] = more
    return s


def prepare(case, seed):
    if case["op"] == "adjust":
        return _prepare_adjust(case, seed)
    dev, g, host = _generators(seed)
    B, page, D = case["B"], case["page"], case["dim"]
    hq, hk = case["q_heads"], case["kv_heads"]
    w, ctx = _sizes(case)
    w = [w[i] for i in torch.randperm(B, generator=host).tolist()]
    ctx = [ctx[i] for i in torch.randperm(B, generator=host).tolist()]
    prefix = [0] * B
    s = {"case": case}
    if case["op"] == "shared":
        p = _prefixes(case)
        p = [p[i] for i in torch.randperm(len(p), generator=host).tolist()]
        each = B // len(p)
        prefix = [p[b // each] for b in range(B)]
        i32 = dict(dtype=torch.int32, device=dev)
        s.update(group_cu=torch.arange(0, B + 1, each, **i32), prefix=torch.tensor(p, **i32),
                 group=torch.arange(B, device=dev) // each)
    # a request's own pages follow those of its group's prefix
    mine = [-(-(c + n) // page) for c, n in zip(ctx, w)]
    most = sum(-(-(c + case["w_hi"]) // page) for c in ctx)       # whatever windows meet them
    front = sum(p // page for p in p) if case["op"] == "shared" else 0
    n_pages = most + front + 3
    order = torch.randperm(n_pages, generator=host).to(torch.int32)
    table = torch.zeros(B, max(p // page + n for p, n in zip(prefix, mine)), dtype=torch.int32)
    k = 0
    for b in range(B):
        f = prefix[b] // page
        if b == 0 or case["op"] != "shared" or b % (B // case["groups"]) == 0:
            table[b, :f] = order[k:k + f]
            k += f
        else:
            table[b, :f] = table[b - 1, :f]
        table[b, f:f + mine[b]] = order[k:k + mine[b]]
        k += mine[b]
    M = sum(w)
    rows = -(-M // PAD) * PAD
    cu, _, _ = _packed(w, rows, dev)
    lengths = torch.tensor([p + c for p, c in zip(prefix, ctx)], dtype=torch.int32)
    s.update(M=M, rows=rows, table=table.to(dev), lengths=lengths.to(dev), cu_seqlens=cu,
             status=torch.zeros(1, dtype=torch.int32, device=dev))
    # the cache as earlier steps left it: blocks of differing magnitude, scales a power of two
    # that keeps each block within e4m3's range
    for name in ("k", "v"):
        x = torch.randn(n_pages, hk, page, D, generator=g, device=dev)
        x *= torch.exp2(torch.rand(n_pages, hk, 1, 1, generator=g, device=dev) * 2 - 1)
        scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(2, 3)) / 448.0)))
        s[name + "_scale"] = scale
        s[name] = (x / scale[:, :, None, None]).to(FP8)
        del x
    s["q"] = torch.randn(rows, hq, D, generator=g, device=dev).to(torch.bfloat16)
    # a stale slot may hold anything: the slots after a request's last token are NaN codes
    for b in range(min(B, 4)):
        used = ctx[b] + w[b] - (mine[b] - 1) * page
        last = int(table[b, prefix[b] // page + mine[b] - 1])
        s["k"].view(torch.uint8)[last, :, used:] = 0x7F
        s["v"].view(torch.uint8)[last, :, used:] = 0x7F
    s["out"] = torch.zeros(rows, hq, D, dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.zeros(rows, hq, dtype=torch.float32, device=dev)
    if case["op"] == "shared":      # two parts per row and head in fp32, and some more
        size = WORKSPACE_BYTES + rows * hq * (D + 1) * 4 + 4096 * (B + 1)
    else:
        size = WORKSPACE_BYTES
    s["workspace"] = torch.empty(size, dtype=torch.uint8, device=dev)
    return s


# ---- the plain forms ---------------------------------------------------------------------
def _plain_adjust(s):
    c, M, more = s["case"], s["M"], s["more"]
    V, dev = c["V"], s["logits"].device
    req, i = s["row_req"][:M].long(), s["row_pos"][:M].long()
    x = s["logits"][:M].float()
    if c["penalties"]:
        ids, at = more["history"].long().clamp(min=0), torch.arange(more["history"].shape[1], device=dev)
        live = at < more["history_len"][:, None]
        answer = (live & (at >= more["prompt_len"][:, None])).float()
        zeros = torch.zeros(c["B"], V, device=dev)
        count = zeros.scatter_add(1, ids, answer)[req]
        drafts = s["block_tokens"].long()[req]
        before = torch.arange(drafts.shape[1], device=dev)[None, :]
        before = ((before >= 1) & (before <= i[:, None])).float()
        count.scatter_add_(1, drafts, before)
        seen = (zeros.scatter_add(1, ids, live.float())[req] > 0) | (count > 0)
        rep = more["repetition"][req, None]
        x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
        x = x - more["frequency"][req, None] * count
        x = x - more["presence"][req, None] * (count > 0)
    if c["bias"]:
        n = torch.arange(c["bias"], device=dev) < more["bias_len"][:, None]
        bias = torch.zeros(c["B"], V, device=dev)
        bias.scatter_add_(1, more["bias_tokens"].long(), torch.where(n, more["bias_values"], 0.0))
        x = x + bias[req]
    if c["masked"]:
        v = torch.arange(V, device=dev)
        allowed = (more["mask"][:M][:, v >> 5] >> (v & 31).to(torch.int32)) & 1
        x = torch.where((allowed == 0) & (more["mask_row"][:M, None] >= 0), -math.inf, x)
    s["out"][:M] = x.to(s["out"].dtype)
    return s["out"]


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
    if c["op"] == "sinks":
        seen &= (t[None, None, :] > pos[:, :, None] - c["window"]) | (t < c["sinks"])[None, None, :]
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
        return _plain_adjust(s) if s["case"]["op"] == "adjust" else _plain_attend(s)
    if "call" not in s:
        s["call"] = _call(s)       # checked and marshalled once for these buffers
    s["call"]()
    return s["out"] if s["case"]["op"] == "adjust" else (s["out"], s["lse"])


def _call(s):
    """The library's prepared call on a state's buffers, as a decode loop keeps it."""
    from speculative_decoding_ragged_gb300 import _binding as bd
    c = s["case"]
    if c["op"] == "adjust":
        return bd.dspark_adjust(s["logits"], s["out"], s["block_tokens"],
                                bd.Adjustments(**s["more"]), cu_seqlens=s["cu_seqlens"],
                                status=s["status"], prepare=True)
    cache = bd.PagedCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"])
    at = (cache, s["q"], s["out"], s["cu_seqlens"], s["lengths"])
    more = dict(lse=s["lse"], status=s["status"], prepare=True)
    if c["op"] == "sinks":
        return bd.dspark_attend_sinks(*at, s["workspace"], window=c["window"], sinks=c["sinks"],
                                      **more)
    return bd.dspark_attend_shared(*at, s["group_cu"], s["prefix"], s["workspace"], **more)


# ---- 64 bits -----------------------------------------------------------------------------
def _exact_adjust(s):
    """Request by request: each token's uses counted, then the formula, row by row."""
    c, more = s["case"], s["more"]
    V, dev = c["V"], s["logits"].device
    cu = s["cu_seqlens"].tolist()
    out = s["out"].double()
    bit = torch.arange(32, device=dev, dtype=torch.int32)
    for b in range(c["B"]):
        prompt = answer = torch.zeros(V, dtype=torch.int64, device=dev)
        if c["penalties"]:
            n, p = int(more["history_len"][b]), int(more["prompt_len"][b])
            h = more["history"][b, :n].long()
            prompt, answer = (torch.bincount(x, minlength=V) for x in (h[:p], h[p:]))
        bias = torch.zeros(V, dtype=torch.float64, device=dev)
        if c["bias"]:
            n = int(more["bias_len"][b])
            bias[more["bias_tokens"][b, :n].long()] = more["bias_values"][b, :n].double()
        for r in range(cu[b], cu[b + 1]):
            x = s["logits"][r].double()
            if c["penalties"]:
                drafts = s["block_tokens"][b, 1:r - cu[b] + 1].long()
                uses = answer + torch.bincount(drafts, minlength=V)
                rep = more["repetition"][b].double()
                again = (uses + prompt) > 0
                x = x * torch.where(again, torch.where(x > 0, 1.0 / rep, rep), torch.ones_like(x))
                x -= uses.double() * more["frequency"][b].double()
                x -= uses.clamp(max=1).double() * more["presence"][b].double()
            x = x + bias
            if c["masked"] and int(more["mask_row"][r]) >= 0:
                words = more["mask"][int(more["mask_row"][r])]
                allowed = ((words[:, None] >> bit) & 1).flatten()[:V].bool()
                x[~allowed] = -math.inf
            out[r] = x
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adjust":
        return _exact_adjust(s)
    if work(case)["flops"] > 3e12:      # FP64 is slow on this part
        return None
    cu, lengths = s["cu_seqlens"].tolist(), s["lengths"].tolist()
    page, D, hk = case["page"], case["dim"], case["kv_heads"]
    group = case["q_heads"] // hk
    out, lse = s["out"].double(), s["lse"].double()
    for b in range(case["B"]):
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
        if case["op"] == "sinks":
            hide = hide | ((t <= pos - case["window"]) & (t >= case["sinks"]))
        score = torch.einsum("whgd,htd->hgwt", q, k) / math.sqrt(D)
        score = score.masked_fill(hide, -math.inf)
        lse[cu[b]:cu[b + 1]] = torch.logsumexp(score, -1).permute(2, 0, 1).reshape(w, -1)
        p = torch.softmax(score, -1)
        out[cu[b]:cu[b + 1]] = torch.einsum("hgwt,htd->whgd", p, v).reshape(w, -1, D)
    return out, lse
