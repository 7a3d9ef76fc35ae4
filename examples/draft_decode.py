"""Serving a pair of layers, one KDA and one softmax attention, with drafted tokens.

Each step a request runs a tree of drafted tokens through both layers at once, one path of it
is accepted, and the rest is dropped: the tree's keys and values are appended to the paged
cache, the KDA pre-step, the recurrence and the attention give every node's outputs, and then
the accepted path's state, convolution inputs, keys and values are kept and the pages behind
them given back.  Halfway, one request forks: another row goes on from what it holds, sharing
its full pages.  Projections and trees are synthetic, and which node is accepted is drawn.

What is checked: the accepted tokens' KDA outputs and states against the same tokens decoded
one by one, and their attention outputs against a plain softmax over the tokens kept so far.

    python examples/draft_decode.py            # needs the built library and a GB300
"""
from __future__ import annotations

import os
import random
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_33_gb300 as kda  # noqa: E402

DEV = "cuda"


def ints(xs):
    return torch.tensor(xs, dtype=torch.int32, device=DEV)


class Server:
    """Two layers' memory, the lists that place tokens in it, and the same KDA layer token by token."""

    def __init__(self, batch, kda_heads, q_heads, kv_heads, head_dim, page_size, num_pages, max_pages,
                 max_nodes, seed=0):
        self.gen = torch.Generator(device=DEV).manual_seed(seed)
        self.rng = random.Random(seed)
        self.batch, self.page_size, self.num_pages, self.max_nodes = batch, page_size, num_pages, max_nodes
        self.H, self.q_heads, self.kv_heads, self.head_dim = kda_heads, q_heads, kv_heads, head_dim
        C = kda_heads * 128
        self.taps = [torch.randn(C, 4, device=DEV, generator=self.gen) * 0.5 for _ in range(3)]
        self.states = torch.zeros(batch, kda_heads, 128, 128, device=DEV)
        self.carried = torch.zeros(batch, 3, 3, C, dtype=torch.bfloat16, device=DEV)
        self.cache = kda.PagedCache(*(torch.zeros(num_pages, page_size, kv_heads, head_dim,
                                                  dtype=torch.bfloat16, device=DEV) for _ in range(2)))
        self.table = torch.full((batch, max_pages), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(num_pages, device=DEV, generator=self.gen).to(torch.int32)
        self.shares = torch.zeros(num_pages, dtype=torch.int32, device=DEV)
        self.kept = [[] for _ in range(batch)]         # keys and values of the tokens kept
        self.plain_states, self.plain_carried = self.states.clone(), self.carried.clone()

    def normal(self, *shape):
        return torch.randn(*shape, device=DEV, generator=self.gen)

    def inputs(self, n):
        """A step's projections: of the KDA layer, its gates, and of the attention layer."""
        x = [self.normal(n, self.H * 128).to(torch.bfloat16) for _ in range(3)]
        g = -torch.nn.functional.softplus(self.normal(n, self.H, 128) - 4.0)
        beta = torch.sigmoid(self.normal(n, self.H))
        q = self.normal(n, self.q_heads, self.head_dim).to(torch.bfloat16)
        k, v = (self.normal(n, self.kv_heads, self.head_dim).to(torch.bfloat16) for _ in range(2))
        return x, g, beta, q, k, v

    def heads(self, xs):
        return [x.view(-1, self.H, 128) for x in xs]

    def place(self, new_lens, k, v):
        """Finds places for the step's tokens and writes their keys and values."""
        seq_lens, cu, slots, used = kda.page_plan(self.lens, ints(new_lens), self.free, self.table,
                                                  self.page_size, self.num_pages, sum(new_lens))
        self.free = self.free[int(used):]
        kda.kda_paged_append(k, v, slots, self.cache)
        return seq_lens, cu

    def prompts(self, new_lens):
        x, g, beta, _, k, v = self.inputs(sum(new_lens))
        self.lens, cu = self.place(new_lens, k, v)
        at = 0
        for b, n in enumerate(new_lens):
            self.kept[b] = [(k[i], v[i]) for i in range(at, at + n)]
            at += n
        *qkv, self.carried = kda.short_conv(*x, *self.taps, cu_seqlens=cu, conv_state=self.carried)
        _, self.states = kda.prefill(*self.heads(qkv), g, beta, cu_seqlens=cu, initial_state=self.states)
        self.plain_states, self.plain_carried = self.states.clone(), self.carried.clone()

    def step(self, sizes):
        """Drafted trees of `sizes` nodes; returns the largest errors of the accepted tokens' KDA
        outputs and attention outputs, relative."""
        parents = [[self.rng.randrange(max(-1, i - 4), i) for i in range(n)] for n in sizes]
        words = torch.cat([kda.ancestor_words(p, DEV) for p in parents])
        last = [self.rng.randrange(-1, n) for n in sizes]
        x, g, beta, q, k, v = self.inputs(sum(sizes))
        seq_lens, cu = self.place(sizes, k, v)
        tree = (cu, words, self.max_nodes)
        qkv = self.heads(kda.short_conv_tree(*x, *self.taps, self.carried, *tree))
        o, u = kda.recurrent_tree_decode(*qkv, g, beta, self.states, *tree, o_dtype=torch.float32)
        attended, _ = kda.paged_tree_decode(q, self.cache, self.table, seq_lens, *tree,
                                            scale=self.head_dim ** -0.5)
        # one node of each tree is accepted, with the path to it
        kda.kda_recurrent_tree_commit(qkv[1], g, u, self.states, None, cu, words, ints(last), self.max_nodes)
        kda.kda_short_conv_tree_commit(*x, self.carried, None, cu, words, ints(last), self.max_nodes)
        self.lens = kda.paged_compact(self.cache, self.table, seq_lens, cu, words, ints(last), self.max_nodes)
        self.release(seq_lens, self.lens)

        paths, at = [], 0                              # rows of the accepted tokens
        for b, n in enumerate(sizes):
            path, i = [], last[b]
            while i >= 0:
                path.insert(0, at + i)
                i = parents[b][i]
            paths.append(path)
            at += n
        return self.check_kda(paths, x, g, beta, o), self.check_attention(paths, q, k, v, attended)

    def release(self, seq_lens, kept_lens):
        freed, num = kda.page_release(seq_lens, kept_lens, self.table, self.page_size, self.shares)
        self.free = torch.cat([self.free, freed[:int(num)]])

    def fork(self, src, dst):
        """Row dst goes on from what request src holds."""
        copies, used = kda.page_fork(ints([src]), ints([dst]), self.lens, self.free, self.table,
                                     self.page_size, self.shares)
        self.free = self.free[int(used):]
        kda.kda_paged_copy(copies, self.cache)
        for memory in (self.states, self.carried, self.plain_states, self.plain_carried):
            memory[dst] = memory[src]
        self.kept[dst] = list(self.kept[src])

    def end(self, b):
        """Request b is done: its pages are given back, its memory is cleared."""
        kept = self.lens.clone()
        kept[b] = 0
        self.release(self.lens, kept)
        self.lens = kept
        for memory in (self.states, self.carried, self.plain_states, self.plain_carried):
            memory[b] = 0
        self.kept[b] = []

    def check_kda(self, paths, x, g, beta, o):
        """The accepted tokens one by one."""
        worst = 0.0
        for depth in range(max(map(len, paths))):
            here = [b for b, p in enumerate(paths) if len(p) > depth]
            rows, index = [paths[b][depth] for b in here], ints(here)
            qkv = self.heads(kda.short_conv_step(*(t[rows].contiguous() for t in x), *self.taps,
                                                 self.plain_carried, index))
            ref = kda.decode_indexed(*qkv, g[rows].contiguous(), beta[rows].contiguous(), self.plain_states,
                                     index, o_dtype=torch.float32)
            worst = max(worst, float((o[rows] - ref).norm() / ref.norm()))
        if not torch.equal(self.carried, self.plain_carried):
            raise RuntimeError("the carried inputs differ from those of single tokens")
        ref = self.plain_states.norm()
        return max(worst, float((self.states - self.plain_states).norm() / ref))

    def check_attention(self, paths, q, k, v, o):
        worst = 0.0
        for b, path in enumerate(paths):
            for row in path:
                self.kept[b].append((k[row], v[row]))
                ks, vs = (torch.stack([t[i] for t in self.kept[b]]).double() for i in range(2))
                p = torch.einsum("hgd,nhd->hgn", q[row].double().view(self.kv_heads, -1, self.head_dim), ks)
                p = torch.softmax(p * self.head_dim ** -0.5, -1)
                ref = torch.einsum("hgn,nhd->hgd", p, vs).reshape(self.q_heads, self.head_dim)
                worst = max(worst, float((o[row].double() - ref).norm() / ref.norm()))
        return worst


def serve(steps=10, max_nodes=24, seed=0):
    """Runs the loop; returns the largest relative errors (KDA outputs and states, attention)."""
    s = Server(batch=6, kda_heads=2, q_heads=8, kv_heads=2, head_dim=128, page_size=16, num_pages=120,
               max_pages=20, max_nodes=max_nodes, seed=seed)
    s.prompts([33, 1, 150, 16, 0, 97])                 # the fifth row waits for a request
    active = [True, True, True, True, False, True]
    worst = (0.0, 0.0)
    for step in range(steps):
        if step == steps // 2:
            s.end(3)                                   # one request ends ..
            s.fork(2, 4)                               # .. and another one goes on twice
            active[3], active[4] = False, True
        sizes = [s.rng.randint(1, max_nodes) if a else 0 for a in active]
        worst = tuple(map(max, worst, s.step(sizes)))
    for b in range(s.batch):                           # all pages come back
        s.end(b)
    if sorted(s.free.tolist()) != list(range(s.num_pages)) or int(s.shares.abs().sum()):
        raise RuntimeError("pages were lost")
    if kda.kda_get_last_device_error() != 0:
        raise RuntimeError("a device error was recorded")
    return worst


if __name__ == "__main__":
    print("relative errors: KDA %.1e, attention %.1e" % serve())
