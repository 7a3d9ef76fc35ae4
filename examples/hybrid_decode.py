"""Serving a pair of layers, one KDA and one softmax attention, with continuous batching.

A model of KDA layers with softmax-attention layers between them keeps two kinds
of memory for a request: a KDA state in a slot of a pool, and keys and values in
pages of a cache.  This example runs both through a serving loop on synthetic
projections: prompts are placed and cached (one plan serves every layer), then
the requests decode token by token; one ends, gives its pages and its state slot
back, and another takes its place.  A prompt runs through the KDA layer and its keys
and values are cached; the attention layer's own outputs for it are not computed here,
as the library has that attention for one new token per sequence only.  The attention
outputs are checked against a plain softmax over the keys that were appended.

    python examples/hybrid_decode.py            # needs the built library and a GB300
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_33_gb300 as kda  # noqa: E402

DEV = "cuda"


class Server:
    """Two layers' memory and the lists that place tokens in it."""

    def __init__(self, batch, kda_heads, q_heads, kv_heads, head_dim, page_size, num_pages,
                 max_pages, fp8=False, seed=0):
        self.gen = torch.Generator(device=DEV).manual_seed(seed)
        self.batch, self.page_size, self.num_pages = batch, page_size, num_pages
        self.kda_heads, self.q_heads, self.kv_heads, self.head_dim = kda_heads, q_heads, kv_heads, head_dim
        self.states = torch.zeros(batch, kda_heads, 128, 128, device=DEV)
        dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
        shape = (num_pages, page_size, kv_heads, head_dim)
        scale = torch.full((kv_heads,), 0.02, device=DEV) if fp8 else None
        self.cache = kda.PagedCache(torch.zeros(shape, dtype=dtype, device=DEV),
                                    torch.zeros(shape, dtype=dtype, device=DEV), scale, scale)
        self.table = torch.full((batch, max_pages), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(num_pages, device=DEV, generator=self.gen).to(torch.int32)
        self.kept = [[] for _ in range(batch)]      # what was appended, for the check

    def normal(self, *shape):
        return torch.randn(*shape, device=DEV, generator=self.gen)

    def kda_inputs(self, n):
        q, k, v = (self.normal(n, self.kda_heads, 128) for _ in range(3))
        q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
        g = -torch.nn.functional.softplus(self.normal(n, self.kda_heads, 128) - 4.0)
        beta = torch.sigmoid(self.normal(n, self.kda_heads))
        return [x.to(torch.bfloat16) for x in (q, k, v)] + [g, beta]

    def plan(self, new_lens):
        """Places the step's tokens: pages, slots and offsets, for all layers."""
        new = torch.tensor(new_lens, dtype=torch.int32, device=DEV)
        seq_lens, cu, slots, used = kda.page_plan(self.lens, new, self.free, self.table,
                                                  self.page_size, self.num_pages, sum(new_lens))
        self.free = self.free[int(used):]            # a server that knows the lengths need not ask
        self.lens = seq_lens
        return cu, slots

    def append(self, slots, new_lens):
        """The attention layer's keys and values of the step, as slices of its projection."""
        width = self.kv_heads * self.head_dim
        rows = self.normal(sum(new_lens), (self.q_heads * self.head_dim) + 2 * width).to(torch.bfloat16)
        k = rows[:, -2 * width:-width].view(-1, self.kv_heads, self.head_dim)
        v = rows[:, -width:].view(-1, self.kv_heads, self.head_dim)
        kda.kda_paged_append(k, v, slots, self.cache)
        at = 0
        for b, n in enumerate(new_lens):
            self.kept[b].append((k[at:at + n], v[at:at + n]))
            at += n
        return rows[:, :self.q_heads * self.head_dim].view(-1, self.q_heads, self.head_dim)

    def prompts(self, new_lens):
        """Prompts through the KDA layer, and into the attention layer's cache."""
        cu, slots = self.plan(new_lens)
        q, k, v, g, beta = self.kda_inputs(sum(new_lens))
        _, states = kda.prefill(q, k, v, g, beta, cu_seqlens=cu, initial_state=self.states)
        self.states = states
        self.append(slots, new_lens)

    def decode(self, active):
        """One token for every active request; returns the attention layer's (q, o)."""
        new_lens = [int(a) for a in active]
        _, slots = self.plan(new_lens)
        rows = [b for b in range(self.batch) if active[b]]
        index = torch.tensor(rows, dtype=torch.int32, device=DEV)
        kda.decode_indexed(*self.kda_inputs(len(rows)), self.states, index)
        q = self.append(slots, new_lens)
        at = index.long()
        o, _ = kda.paged_decode(q, self.cache, self.table[at].contiguous(), self.lens[at].contiguous(),
                                self.head_dim ** -0.5)
        return rows, q, o

    def end(self, b):
        """Request b is done: its pages go back to the free list, its memory is cleared."""
        held = -(-int(self.lens[b]) // self.page_size)
        self.free = torch.cat([self.free, self.table[b, :held]])
        self.lens = self.lens.clone()
        self.lens[b] = 0
        self.table[b] = -1
        self.states[b] = 0
        self.kept[b] = []

    def expected(self, b, q):
        """Plain softmax attention of request b's query over all that it appended."""
        k = torch.cat([x[0] for x in self.kept[b]]).double()
        v = torch.cat([x[1] for x in self.kept[b]]).double()
        if self.cache.k_scale is not None:           # what the 8-bit cache holds of them
            s = self.cache.k_scale.double()[:, None]
            k, v = (((x.float() / s.float()).clamp(-448, 448).to(torch.float8_e4m3fn).double()) * s
                    for x in (k, v))
        q = q.double().view(self.kv_heads, -1, self.head_dim)
        p = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k) * self.head_dim ** -0.5, -1)
        return torch.einsum("hgn,nhd->hgd", p, v).reshape(self.q_heads, self.head_dim)


def serve(steps=24, fp8=False, seed=0):
    """Runs the loop; returns the largest relative error of the attention outputs."""
    s = Server(batch=6, kda_heads=4, q_heads=16, kv_heads=4, head_dim=128, page_size=16,
               num_pages=200, max_pages=40, fp8=fp8, seed=seed)
    s.prompts([33, 1, 250, 16, 0, 97])               # the fifth row waits for a request
    active = [True, True, True, True, False, True]
    worst = 0.0
    for step in range(steps):
        if step == steps // 2:
            s.end(2)                                 # a long request ends ..
            s.prompts([0, 0, 70, 0, 45, 0])          # .. and two others begin
            active[4] = True
        rows, q, o = s.decode(active)
        for i, b in enumerate(rows):
            ref = s.expected(b, q[i])
            worst = max(worst, float((o[i].double() - ref).norm() / ref.norm()))
    if kda.kda_get_last_device_error() != 0:
        raise RuntimeError("a device error was recorded")
    if not bool(torch.isfinite(s.states).all()):
        raise RuntimeError("a KDA state is not finite")
    return worst


if __name__ == "__main__":
    for fp8 in (False, True):
        print(f"{'8-bit' if fp8 else 'bf16'} cache: attention outputs within "
              f"{serve(fp8=fp8):.1e} of plain softmax (relative)")
