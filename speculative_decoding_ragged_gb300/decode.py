"""The target forward's ragged operators as one decode step uses them.

CachedAttention is one attention layer over the paged 8-bit cache: it stores the packed rows'
keys and values (dspark_append, which also rotates the queries) and attends over what the cache
then holds (dspark_attend; dspark_attend_sinks where a window keeps its first tokens visible;
dspark_attend_shared where requests share a prefix). All calls size themselves on the device, so
they capture into the same CUDA graph as the rest of the step.

DecodeLoop runs whole steps of a small random model (one attention layer) with
it: draft a block, schedule and pack it, run the target over the packed rows, adjust its logits
(dspark_adjust, if anything is to be), verify, scatter,
advance the lengths. The draft attends within its block only, its queries and keys rotated by
dspark_rotate. `python -m speculative_decoding_ragged_gb300.decode` decodes a few steps and
prints what was accepted.
"""
from __future__ import annotations

from typing import Optional

import numpy as np
import torch

from . import _binding as bd
from .step import DSparkStep


def packed_owners(row_req, cu_seqlens):
    """row_req with -1 in the rows at or past cu_seqlens[B]: dspark_pack leaves those past its tier as
    they were, which is an earlier step's owners."""
    index = torch.arange(row_req.numel(), dtype=torch.int32, device=row_req.device)
    return torch.where(index < cu_seqlens[-1], row_req, -1).to(torch.int32)


class CachedAttention:
    """One layer's cache and the buffers its calls need; `rows` is the most rows of a call.

    Rows at or past cu_seqlens[B] are padding, whatever row_req says of them (dspark_pack leaves
    those past its tier as they were): two small kernels before the calls see to it. Where many
    layers share the rows, `owned=True` spares them: row_req is then packed_owners' already.

    `window` and `sinks` are dspark_attend_sinks', `shared` is dspark_attend_shared's (group_cu,
    prefix), tensors whose values may change between calls."""

    def __init__(self, rows: int, q_heads: int, kv_heads: int, dim: int, table: torch.Tensor,
                 n_pages: int, page: int, rope: Optional[bd.Rope] = None, *, window: int = 0,
                 sinks: int = 0, shared=None, dtype=torch.bfloat16):
        if sinks and not window:
            raise ValueError("sinks need a window: without one every token is visible")
        if shared is not None and window:
            raise ValueError("a shared prefix has no window")
        self.cache = bd.PagedCache.empty(n_pages, kv_heads, page, dim, table)
        self.rope, self.window, self.sinks, self.shared = rope, window, sinks, shared
        dev = table.device
        self.turned = torch.zeros(rows, q_heads, dim, dtype=dtype, device=dev)
        self.out = torch.zeros(rows, q_heads, dim, dtype=dtype, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.owners = torch.full((rows,), -1, dtype=torch.int32, device=dev)
        self.index = torch.arange(rows, dtype=torch.int32, device=dev)
        self.live = torch.zeros(rows, dtype=torch.bool, device=dev)
        self.nobody = torch.tensor(-1, dtype=torch.int32, device=dev)
        need = bd.dspark_attend_workspace_bytes(kv_heads, dim) if shared is None else \
            bd.dspark_attend_shared_workspace_bytes(rows, q_heads, kv_heads, dim, table.shape[0])
        self.workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)

    def prepare(self, q, k, v, row_req, row_pos, cu_seqlens, lengths, *, owned=False):
        """The calls for these tensors (which stay alive and in place), checked once."""
        rows = q.shape[0]
        turned, out = self.turned[:rows], self.out[:rows]
        calls = []
        if not owned:
            given, last = row_req[:rows], cu_seqlens[-1:]
            row_req, index, live = self.owners[:rows], self.index[:rows], self.live[:rows]

            def owners():
                torch.lt(index, last, out=live)
                torch.where(live, given, self.nobody, out=row_req)
            calls.append(owners)
        calls.append(bd.dspark_append(self.cache, k, v, row_req, row_pos, lengths, rope=self.rope, q=q,
                                      q_out=turned, status=self.status, prepare=True))
        what = (self.cache, turned, out, cu_seqlens, lengths)
        more = dict(status=self.status, prepare=True)
        if self.shared is not None:
            attend = bd.dspark_attend_shared(*what, *self.shared, self.workspace, **more)
        elif self.sinks:
            attend = bd.dspark_attend_sinks(*what, self.workspace, window=self.window, sinks=self.sinks,
                                            **more)
        else:
            attend = bd.dspark_attend(*what, self.workspace, window=self.window, **more)
        return calls + [attend]

    def run(self, q, k, v, row_req, row_pos, cu_seqlens, lengths, *, owned=False):
        """Packed rows in, attention out ([rows, q_heads, dim], overwritten by the next call);
        lengths: tokens in the cache before these rows."""
        for call in self.prepare(q, k, v, row_req, row_pos, cu_seqlens, lengths, owned=owned):
            call()
        return self.out[:q.shape[0]]


class DecodeLoop:
    """`prompt` tokens (whole pages; self.prompt) stand before every request's own, in the same pages;
    `repetition`, `presence`, `frequency` (one number for all requests) and `mask` (a grammar's allowed
    tokens, [words] int32, for every row) are dspark_adjust's. A loop that adjusts keeps whole histories in
    step.out_tokens: the prompt, the first anchor, then what is committed; any other what is committed."""

    def __init__(self, B: int, gamma: int, V: int, *, width: int = 256, q_heads: int = 8,
                 kv_heads: int = 2, dim: int = 64, page: int = 16, max_len: int = 512,
                 window: int = 0, sinks: int = 0, prompt: int = 0, repetition: float = 1.0,
                 presence: float = 0.0, frequency: float = 0.0, mask: Optional[torch.Tensor] = None,
                 seed: int = 0, device="cuda"):
        self.B, self.gamma, self.V = B, gamma, V
        self.q_heads, self.kv_heads, self.dim = q_heads, kv_heads, dim
        dev = torch.device(device)
        gen = torch.Generator().manual_seed(seed)

        def weight(*shape):
            w = torch.randn(*shape, generator=gen) * shape[0] ** -0.5
            return w.to(dev, torch.bfloat16)

        qkv = (q_heads + 2 * kv_heads) * dim
        self.emb = weight(V, width) * V ** 0.5
        self.w_qkv, self.w_out, self.w_head = weight(width, qkv), weight(q_heads * dim, width), weight(width, V)
        # the draft: its slots' embeddings; it shares the target's projections
        self.slot = weight(gamma, width) * (0.1 * gamma ** 0.5)

        blocks = -(-(max_len + gamma) // page)
        table = torch.randperm(B * blocks, generator=gen).to(torch.int32).view(B, blocks).to(dev)
        if prompt % page:
            raise ValueError(f"a prompt of {prompt} tokens does not fill whole pages of {page}")
        front = B * blocks + torch.arange(prompt // page, dtype=torch.int32, device=dev)
        table = torch.cat([front.repeat(B, 1), table], 1).contiguous()
        i32 = dict(dtype=torch.int32, device=dev)
        shared = (torch.tensor([0, B], **i32), torch.tensor([prompt], **i32)) if prompt else None
        self.rope = bd.Rope.make(dim, device=dev)
        tiers = sorted({B, B * (gamma + 1) // 2, B * gamma})
        adjusts = (repetition, presence, frequency) != (1.0, 0.0, 0.0) or mask is not None
        before = prompt + 1 if adjusts else 0                # tokens of a history that no step commits
        self.step = DSparkStep(B, gamma, V, tiers, 1.0, 1e-3 * np.arange(B + 1),
                               1e-3 * np.arange(B * gamma + 1), out_cap=before + max_len, device=dev)
        self.attention = CachedAttention(self.step.packed_cap, q_heads, kv_heads, dim, table,
                                         B * blocks + front.numel(), page, self.rope, window=window,
                                         sinks=sinks, shared=shared)
        self.lengths = torch.full((B,), prompt, **i32)
        self.anchor = torch.randint(V, (B,), generator=gen, dtype=torch.int32).to(dev)
        self.slots = torch.arange(gamma, **i32)
        self.prompt = torch.randint(V, (prompt,), generator=gen).to(dev)
        if prompt:
            self.fill(self.prompt)
        self.how = None
        if adjusts:
            self.step.out_tokens[:, :prompt] = self.prompt
            self.step.out_tokens[:, prompt] = self.anchor
            self.step.out_len.fill_(before)
            each = lambda x: torch.full((B,), x, dtype=torch.float32, device=dev)    # noqa: E731
            rows = torch.zeros(self.step.packed_cap, **i32) if mask is not None else None
            self.how = bd.Adjustments(
                history=self.step.out_tokens, history_len=self.step.out_len,
                prompt_len=torch.full((B,), prompt, **i32), repetition=each(repetition),
                presence=each(presence), frequency=each(frequency),
                mask=mask[None] if mask is not None else None, mask_row=rows)

    def fill(self, tokens):
        """The shared prompt's keys and values, stored once, as request 0's tokens."""
        _, k, v = self.project(self.emb[tokens])
        at = torch.arange(tokens.numel(), dtype=torch.int32, device=tokens.device)
        bd.dspark_append(self.attention.cache, k, v, torch.zeros_like(at), at,
                         torch.zeros_like(self.lengths), rope=self.rope, status=self.attention.status)

    def project(self, x):
        """[rows, width] -> q, k, v, each [rows, heads, dim]: slices of one product."""
        y = x @ self.w_qkv
        a, b = self.q_heads * self.dim, (self.q_heads + self.kv_heads) * self.dim
        return (y[:, :a].unflatten(1, (self.q_heads, self.dim)),
                y[:, a:b].unflatten(1, (self.kv_heads, self.dim)),
                y[:, b:].unflatten(1, (self.kv_heads, self.dim)))

    def draft(self):
        """A block per request: its anchor, then gamma - 1 proposals and their confidences."""
        B, G = self.B, self.gamma
        x = (self.emb[self.anchor.long()][:, None] + self.slot).flatten(0, 1)
        q, k, v = self.project(x)
        positions = (self.lengths[:, None] + self.slots).flatten()
        rotated = []
        for t in (q, k):
            y = torch.empty(t.shape, dtype=t.dtype, device=t.device)
            bd.dspark_rotate(t, y, positions, self.rope)
            rotated.append(y)
        group = self.q_heads // self.kv_heads
        q, k, v = (t.unflatten(0, (B, G)).transpose(1, 2) for t in (*rotated, v))
        k, v = (t.repeat_interleave(group, 1) for t in (k, v))
        o = torch.softmax(q.float() @ k.float().mT * self.dim ** -0.5, -1) @ v.float()
        x = x + o.transpose(1, 2).reshape(B * G, -1).to(x.dtype) @ self.w_out
        top = torch.softmax((x @ self.w_head).float(), -1).max(-1)
        tokens = torch.cat([self.anchor[:, None],
                            top.indices.view(B, G)[:, :G - 1].to(torch.int32)], 1)
        return tokens.contiguous(), top.values.view(B, G)[:, :G - 1].contiguous()

    def target(self):
        """Logits of the packed rows, their keys and values stored on the way."""
        s = self.step
        x = self.emb[s.packed_ids.clamp(0, self.V - 1).long()]
        o = self.attention.run(*self.project(x), s.row_req, s.row_pos, s.cu, self.lengths)
        return (x + o.flatten(1) @ self.w_out) @ self.w_head

    def advance(self):
        """The accepted rows stay in the cache; the next step's rows overwrite the others'."""
        L = self.step.accept_len
        self.lengths += L
        self.anchor = self.step.committed.gather(1, (L - 1).clamp(min=0)[:, None].long())[:, 0]

    def run(self):
        """One step: every request commits one to gamma tokens."""
        tokens, conf = self.draft()
        self.step.schedule_pack(conf, tokens)
        logits = self.target()
        if self.how is not None:
            self.step.adjust(logits, tokens, self.how)
        self.step.verify_scatter(logits, tokens)
        self.advance()


def main():
    for what, more in (("plain", dict()), ("a window of 32 and 4 sinks", dict(window=32, sinks=4)),
                       ("a shared prompt and penalties", dict(prompt=512, repetition=1.2, frequency=0.5))):
        loop = DecodeLoop(8, 4, 2048, **more)
        print(what)
        for i in range(8):
            loop.run()
            L = loop.step.accept_len.tolist()
            print(f"step {i}: windows {loop.step.windows.tolist()} committed {L}")
        print("lengths", loop.lengths.tolist(), "status",
              int(loop.step.status.item()) | int(loop.attention.status.item()))


if __name__ == "__main__":
    main()
