"""The operators of a step of drafted tokens, and those that share, move and free pages, as
measured cases: each in its plain form (elementary torch operations) and as the calls a user
makes.

A serving loop that drafts runs, for every request, a small tree of drafted tokens through the
layers at once: ``conv`` and ``recur`` in a KDA layer, ``attend`` in a softmax-attention layer,
whose keys and values the paged cache already holds; then ``accept`` keeps one path of the tree
in both kinds of memory.  ``pages`` forks requests and frees what ended ones held.

A tree is given by one 64-bit word for each node: bit j is set where the node sees node j of its
request (its ancestors, and itself).
"""
import math
import random

import torch

own = False

DEV = "cuda"


# --- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # one request with eight drafted tokens in a short conversation: latency
        dict(name="attend_b1_n8", op="attend", B=1, nlo=8, nhi=8, lo=301, hi=301, Hkv=8, G=4, D=128,
             page=16, cache="bf16", order="token", mix=1),
        # a serving batch with sixteen drafted tokens each, ragged contexts
        dict(name="attend_b32_n16", op="attend", B=32, nlo=16, nhi=16, lo=500, hi=6000, Hkv=8, G=8,
             D=128, page=16, cache="bf16", order="token", mix=2),
        # an 8-bit cache, odd trees of every size up to 21 nodes
        dict(name="attend_b64_fp8", op="attend", B=64, nlo=1, nhi=21, lo=1000, hi=8192, Hkv=8, G=8,
             D=128, page=64, cache="fp8", order="head", mix=3),
        # the widest trees at 96 query heads: as much arithmetic as memory
        dict(name="attend_b12_n64_g12", op="attend", B=12, nlo=64, nhi=64, lo=700, hi=9001, Hkv=8, G=12,
             D=128, page=24, cache="bf16", order="token", mix=4),
        # the KDA layer of two requests, a few drafted tokens: latency
        dict(name="recur_b2_n5", op="recur", B=2, nlo=5, nhi=5, H=96, state="fp32", out="bf16", chain=False,
             mix=5),
        # the KDA layer of a serving batch at 96 heads
        dict(name="recur_b64_n16", op="recur", B=64, nlo=7, nhi=16, H=96, state="fp32", out="bf16",
             chain=False, mix=6),
        # the pre-step of the same layer for a small batch
        dict(name="conv_b4_n8", op="conv", B=4, nlo=8, nhi=8, H=96, chain=False, mix=7),
        # and for many requests with odd trees
        dict(name="conv_b128_n33", op="conv", B=128, nlo=9, nhi=33, H=96, chain=False, mix=8),
        # what follows a verified step of a small batch in a KDA and an attention layer
        dict(name="accept_b4_n8", op="accept", B=4, nlo=8, nhi=8, H=96, state="bf16", lo=100, hi=2000, Hkv=8,
             D=128, page=16, cache="bf16", order="token", mix=9),
        # and of a serving batch with an fp32 state pool
        dict(name="accept_b64_n16", op="accept", B=64, nlo=5, nhi=16, H=96, state="fp32", lo=100, hi=3000,
             Hkv=8, D=128, page=32, cache="bf16", order="head", mix=10),
        # four continuations begin, they and some others end
        dict(name="pages_b16_f4", op="pages", B=16, forks=4, lo=50, hi=900, Hkv=8, D=128, page=16,
             cache="bf16", mix=11),
        # a large pool: 300 branches begin, they and a third of the others end
        dict(name="pages_b1024_f300", op="pages", B=1024, forks=300, lo=20, hi=1500, Hkv=8, D=128, page=16,
             cache="bf16", mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "recur", "recur", "conv", "accept", "accept", "pages"])
    mix = rng.randrange(1 << 30)
    nhi = rng.choice([1, 2, 3, 5, 8, 12, 16, 21, 32, 47, 64])
    nlo = rng.choice([1, nhi, max(1, nhi // 2)])
    page = rng.choice([16, 16, 24, 32, 64, 64, 128])
    Hkv, D = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128, 128, 256])
    cache, order = rng.choice(["bf16", "bf16", "fp8"]), rng.choice(["token", "head"])
    chain = rng.random() < 0.25
    if op == "attend":
        G = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24])
        B = _log_int(rng, 1, 64)
        # keys of all requests together, by what they read and by what they compute
        most = min(240000 * 8 * 128 // (Hkv * D), 12 * 9000 * 64 * 12 * 8 * 128 // (nhi * G * Hkv * D))
        hi = nhi + _log_int(rng, 1, max(1, min(65536, most // B)))
        return dict(op=op, B=B, nlo=nlo, nhi=nhi, lo=max(nhi, hi // rng.choice([1, 2, 16])), hi=hi, Hkv=Hkv,
                    G=G, D=D, page=page, cache=cache, order=order, mix=mix)
    if op == "pages":
        B = _log_int(rng, 2, 1024)
        forks = _log_int(rng, 1, max(1, B // 3))
        hi = _log_int(rng, 2, max(2, min(20000, 1000000 * 8 * 128 // (B * Hkv * D))))
        return dict(op=op, B=B, forks=forks, lo=max(1, hi // 16), hi=hi, Hkv=Hkv, D=D, page=page, cache=cache,
                    mix=mix)
    H = rng.choice([1, 4, 16, 32, 96])
    most = max(1, min(64, 64 * 96 * 16 // (H * nhi)))
    B = _log_int(rng, 1, most)
    if op == "conv":
        return dict(op=op, B=B, nlo=nlo, nhi=nhi, H=H, chain=chain, mix=mix)
    state = rng.choice(["fp32", "bf16"])
    if op == "recur":
        return dict(op=op, B=B, nlo=nlo, nhi=nhi, H=H, state=state, out=rng.choice(["bf16", "bf16", "fp32"]),
                    chain=chain, mix=mix)
    hi = nhi + _log_int(rng, 1, 3000)
    return dict(op=op, B=B, nlo=nlo, nhi=nhi, H=H, state=state, lo=max(nhi, hi // 8), hi=hi, Hkv=Hkv, D=D,
                page=page, cache=cache, order=order, mix=mix)


def _pages(n, ps):
    return -(-n // ps)


def _trees(case):
    """Node counts and the nodes' parents (-1: the context), the same for every seed."""
    rng = random.Random(case["mix"])
    trees = []
    for _ in range(case["B"]):
        n = rng.randint(case["nlo"], case["nhi"])
        # node 0 is the token that was sampled last; drafts branch from any node, mostly a late one
        trees.append([-1] + [i - 1 if case.get("chain") or rng.random() < 0.5 else rng.randrange(i)
                             for i in range(1, n)])
    return trees


def _words(parents):
    words = []
    for i, p in enumerate(parents):
        words.append((words[p] if p >= 0 else 0) | 1 << i)
    return words


def _lens(case):
    """The lengths of a case's requests, the drafted tokens included."""
    rng = random.Random(case["mix"] + 1)
    lo, hi = case["lo"], case["hi"]
    if hi <= 8 * lo:
        return [rng.randint(lo, hi) for _ in range(case["B"])]
    return [_log_int(rng, lo, hi) for _ in range(case["B"])]


def _last(case):
    """The last node of each request's accepted path; a few requests keep nothing."""
    rng = random.Random(case["mix"] + 2)
    return [-1 if rng.random() < 0.06 else rng.randrange(len(t)) for t in _trees(case)]


def _ends(case):
    """Of a case of pages: the forks, and the lengths that the requests keep afterwards."""
    rng = random.Random(case["mix"] + 3)
    B, forks = case["B"], min(case["forks"], case["B"] - 1)
    rows = list(range(B))
    rng.shuffle(rows)
    dst, others = rows[:forks], rows[forks:]
    src = [rng.choice(others) for _ in dst]
    lens = _lens(case)
    for d in dst:
        lens[d] = 0
    grown = list(lens)
    for s, d in zip(src, dst):
        grown[d] = lens[s]
    # a third ends, and all that was forked (so a pass can be repeated); some lose their last
    # tokens, the others go on
    ended = set(dst)
    kept = [0 if b in ended or rng.random() < 0.33
            else n - rng.randint(0, min(n, 40)) if rng.random() < 0.3 else n
            for b, n in enumerate(grown)]
    return src, dst, lens, grown, kept


# --- inputs --------------------------------------------------------------------------------

def _pool(num_pages, page, Hkv, D, cache, order, gen, sigma):
    """A cache [num_pages, page, Hkv, D] (a view where the pages are stored head by head)."""
    dtype = torch.float8_e4m3fn if cache == "fp8" else torch.bfloat16
    shape = (num_pages, Hkv, page, D) if order == "head" else (num_pages, page, Hkv, D)
    t = torch.zeros(shape, dtype=dtype, device=DEV)
    for i in range(0, num_pages, 4096):  # in parts: the fp32 draw of a whole pool would be large
        part = t[i:i + 4096]
        part.copy_((torch.randn(part.shape, device=DEV, generator=gen) * sigma))
    return t.permute(0, 2, 1, 3) if order == "head" else t


def _table(held, spare, gen):
    """A block table over a shuffled pool, and the pages that are left."""
    num_pages, width = sum(held) + spare, max(max(held), 1)
    order = torch.randperm(num_pages, device=DEV, generator=gen).to(torch.int32)
    h = torch.tensor(held, device=DEV)
    first = torch.cumsum(h, 0) - h
    at = (first[:, None] + torch.arange(width, device=DEV)[None]).clamp(max=num_pages - 1)
    return order[at].contiguous(), order[sum(held):].contiguous(), num_pages


def _signed(words):
    """64-bit words as torch holds them."""
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device=DEV)


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 1000003 + case["mix"] % 99991)
    s = dict(case=case)
    op = case["op"]
    i32 = dict(dtype=torch.int32, device=DEV)

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=gen)

    if op != "pages":
        trees = _trees(case)
        counts = [len(t) for t in trees]
        B, N = case["B"], sum(counts)
        s["nmax"] = max(counts)
        s["cu"] = torch.tensor([sum(counts[:b]) for b in range(B + 1)], **i32)
        s["anc"] = _signed([w for t in trees for w in _words(t)])
    if "Hkv" in case:
        Hkv, D, ps = case["Hkv"], case["D"], case["page"]
        fp8 = case["cache"] == "fp8"
        s["k_scale"] = s["v_scale"] = None
        if fp8:  # a head's scale puts its largest values near the top of the 8-bit range
            s["k_scale"] = 0.01 + 0.02 * torch.rand(Hkv, device=DEV, generator=gen)
            s["v_scale"] = 0.01 + 0.02 * torch.rand(Hkv, device=DEV, generator=gen)
        lens = _ends(case)[2] if op == "pages" else _lens(case)
        s["table"], s["free"], s["num_pages"] = _table(
            [_pages(n, ps) for n in lens], 8 + (case["forks"] if op == "pages" else 0), gen)
        s["seq_lens"] = torch.tensor(lens, **i32)
        order = case.get("order", "token")
        for name in ("k_cache", "v_cache"):
            s[name] = _pool(s["num_pages"], ps, Hkv, D, case["cache"], order, gen, 50.0 if fp8 else 1.0)
        if own:
            import gated_delta_rule_33_gb300 as kda
            s["cache"] = kda.PagedCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if op == "attend":
        Hq = Hkv * case["G"]
        # scores of spread about 2: some keys matter much more than others
        s["q"] = (2.0 * normal(N, Hq, D)).to(torch.bfloat16)
        s["scale"] = D ** -0.5
        s["o"] = torch.empty(N, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(N, Hq, device=DEV)
        if own:
            s["ws"] = torch.empty(max(16, kda.kda_paged_tree_decode_workspace_size(
                B, s["nmax"], Hq, Hkv, D)), dtype=torch.uint8, device=DEV)
        return s
    if op == "pages":
        src, dst, lens, grown, kept = _ends(case)
        table = torch.full((case["B"], max(_pages(n, ps) for n in grown) + 1), -1, **i32)
        table[:, :s["table"].shape[1]] = s["table"]
        s["table"] = table
        s["src"], s["dst"] = torch.tensor(src, **i32), torch.tensor(dst, **i32)
        s["kept"] = torch.tensor(kept, **i32)
        s["shares"] = torch.zeros(s["num_pages"], **i32)
        s["copies"], s["used"] = torch.empty(len(src), 3, **i32), torch.empty(1, **i32)
        s["freed"], s["num_freed"] = torch.full((s["num_pages"],), -1, **i32), torch.empty(1, **i32)
        return s
    H = case["H"]
    slots = torch.randperm(B + 3, device=DEV, generator=gen)[:B].to(torch.int32)
    if op in ("conv", "accept"):
        C = H * 128
        s["x"] = [normal(N, C).to(torch.bfloat16) for _ in range(3)]
        s["conv_pool"] = normal(B + 3, 3, 3, C).to(torch.bfloat16)
        s["slots"] = slots
    if op == "conv":
        s["w"] = [0.5 * normal(C, 4) for _ in range(3)]
        s["y"] = [torch.empty(N, C, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
        return s
    q, k = (_unit(normal(N, H, 128)).to(torch.bfloat16) for _ in range(2))
    s["q"], s["k"], s["v"] = q, k, normal(N, H, 128).to(torch.bfloat16)
    # decays from nearly none to several nats a token, as the gate gives them
    s["g"] = -torch.nn.functional.softplus(2.0 * normal(N, H, 128) - 3.0)
    s["beta"] = torch.sigmoid(normal(N, H))
    s["slots"] = slots
    s["pool"] = torch.empty(B + 3, H, 128, 128, device=DEV,
                            dtype=torch.float32 if case["state"] == "fp32" else torch.bfloat16)
    for i in range(B + 3):
        s["pool"][i].copy_(0.3 * normal(H, 128, 128))
    if op == "recur":
        s["scale"] = 128 ** -0.5
        s["o"] = torch.empty(N, H, 128, device=DEV,
                             dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16)
        s["u"] = torch.empty(N, H, 128, device=DEV)
        return s
    s["u"] = 0.5 * normal(N, H, 128)  # what the layer's step left
    s["last"], s["kept"] = torch.tensor(_last(case), **i32), torch.empty(B, **i32)
    return s


# --- one pass ------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"attend": _plain_attend, "recur": _plain_recur, "conv": _plain_conv,
                "accept": _plain_accept, "pages": _plain_pages}[op](s)
    import gated_delta_rule_33_gb300 as kda
    if op == "attend":
        kda.kda_paged_tree_decode(s["q"], s["cache"], s["table"], s["seq_lens"], s["cu"], s["anc"],
                                  s["nmax"], s["scale"], s["o"], s["lse"], s["ws"])
        return dict(o=s["o"], lse=s["lse"])
    if op == "recur":
        kda.kda_recurrent_tree_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], s["slots"],
                                      s["cu"], s["anc"], s["nmax"], s["scale"], s["o"], s["u"])
        return dict(o=s["o"], u=s["u"])
    if op == "conv":
        kda.kda_short_conv_qkv_tree(*s["x"], *s["w"], s["conv_pool"], s["slots"], s["cu"], s["anc"],
                                    s["nmax"], *s["y"])
        return dict(q=s["y"][0], k=s["y"][1], v=s["y"][2])
    if op == "accept":
        kda.kda_recurrent_tree_commit(s["k"], s["g"], s["u"], s["pool"], s["slots"], s["cu"], s["anc"],
                                      s["last"], s["nmax"])
        kda.kda_short_conv_tree_commit(*s["x"], s["conv_pool"], s["slots"], s["cu"], s["anc"], s["last"],
                                       s["nmax"])
        kda.kda_paged_compact(s["cache"], s["table"], s["seq_lens"], s["cu"], s["anc"], s["last"],
                              s["nmax"], s["kept"])
        return dict(pool=s["pool"], conv_pool=s["conv_pool"], k_cache=s["k_cache"], v_cache=s["v_cache"],
                    kept=s["kept"])
    kda.kda_page_fork(s["src"], s["dst"], s["seq_lens"], s["free"], s["table"], s["case"]["page"],
                      s["shares"], s["copies"], s["used"])
    kda.kda_paged_copy(s["copies"], s["cache"])
    kda.kda_page_release(s["seq_lens"], s["kept"], s["table"], s["case"]["page"], s["shares"], s["freed"],
                         s["num_freed"])
    return dict(table=s["table"], seq_lens=s["seq_lens"], shares=s["shares"], copies=s["copies"],
                used=s["used"], freed=s["freed"], num_freed=s["num_freed"], k_cache=s["k_cache"],
                v_cache=s["v_cache"])


def _raw(cache):
    """A cache whose elements can be indexed: 8-bit ones as bytes."""
    return cache.view(torch.uint8) if cache.element_size() == 1 else cache


def _gather(cache, scale, table, length):
    """The first `length` keys of every request, [B, Hkv, length, D] in 32 bits."""
    x = _raw(cache)[table.long()].view(cache.dtype)
    x = x.flatten(1, 2)[:, :length].permute(0, 2, 1, 3).float()
    return x if scale is None else x * scale[None, :, None, None]


def _padded(s, nmax):
    """Rows of a packed batch as [B, nmax] indices, and which of them exist."""
    cu = s["cu"].long()
    i = torch.arange(nmax, device=DEV)[None]
    real = i < (cu[1:] - cu[:-1])[:, None]
    return torch.where(real, cu[:-1, None] + i, torch.zeros_like(i)), real


def _bits(words, n):
    """Bit j of every word, j < n, as truth values."""
    return (words[..., None] >> torch.arange(n, device=DEV)) & 1 == 1


def _plain_attend(s):
    c = s["case"]
    B, Hkv, G, D, n = c["B"], c["Hkv"], c["G"], c["D"], s["nmax"]
    rows, real = _padded(s, n)
    length = s["table"].shape[1] * c["page"]
    k = _gather(s["k_cache"], s["k_scale"], s["table"], length)
    v = _gather(s["v_cache"], s["v_scale"], s["table"], length)
    counts = (s["cu"][1:] - s["cu"][:-1]).long()
    context = s["seq_lens"].long() - counts
    j = torch.arange(length, device=DEV)[None] - context[:, None]          # the drafted node of a key
    o, lse = torch.empty_like(s["o"]), torch.empty_like(s["lse"])
    some = max(1, min(B, 2 ** 30 // (Hkv * n * G * length)))               # requests at a time
    for b in range(0, B, some):
        e = min(B, b + some)
        q = s["q"][rows[b:e]].float().view(e - b, n, Hkv, G, D) * s["scale"]
        scores = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(e - b, Hkv, n * G, D),
                              k[b:e].transpose(2, 3)).view(e - b, Hkv, n, G, length)
        node = j[b:e, None, :].expand(-1, n, -1)
        word = s["anc"][rows[b:e]][:, :, None]
        seen = (node < 0) | ((node < counts[b:e, None, None]) & ((word >> node.clamp(0, 63)) & 1 == 1))
        scores = torch.where(seen[:, None, :, None, :], scores, torch.full_like(scores, -math.inf))
        m = scores.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        p = torch.exp(scores - m)
        total = p.sum(-1, keepdim=True)
        x = torch.matmul(p.view(e - b, Hkv, n * G, length), v[b:e]).view(e - b, Hkv, n, G, D)
        x = torch.where(total > 0, x / total, torch.zeros_like(x)).permute(0, 2, 1, 3, 4)
        y = (m + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3)
        o[rows[b:e][real[b:e]]] = x.reshape(e - b, n, Hkv * G, D)[real[b:e]].to(o.dtype)
        lse[rows[b:e][real[b:e]]] = y.reshape(e - b, n, Hkv * G)[real[b:e]]
    return dict(o=o, lse=lse)


def _plain_recur(s):
    """Node by node over all requests: each node's state, applied to a vector, is the first
    state behind the decays of its path and one product of every ancestor."""
    n, scale = s["nmax"], s["scale"]
    rows, real = _padded(s, n)
    below = torch.tril(torch.ones(n, n, dtype=torch.bool, device=DEV), -1)
    anc = _bits(s["anc"][rows], n) & below                                 # [B, n, n], strict
    B, H = rows.shape[0], s["q"].shape[1]
    q, k, v = (s[x][rows].float() for x in ("q", "k", "v"))
    g, beta = s["g"][rows], s["beta"][rows]
    S = s["pool"][s["slots"].long()].float()
    u, o = torch.zeros_like(v), torch.zeros_like(v)
    own_node = torch.eye(n, dtype=torch.bool, device=DEV)
    after = torch.triu(torch.ones(n, n, dtype=torch.bool, device=DEV), 1)  # [j, l]: l comes after j
    flat = g.reshape(B, n, -1)
    for i in range(n):
        path = (anc[:, i] | own_node[i]).float()                           # [B, n]
        decay = torch.exp(torch.matmul(path[:, None], flat).view(B, H, 128))
        behind = torch.exp(torch.matmul(path[:, None] * after.float(), flat).view(B, n, H, 128))
        first = torch.matmul(torch.stack([decay * k[:, i], decay * q[:, i]], 2), S)
        ki, qi = ((behind * k * x[:, i, None]).sum(-1) for x in (k, q))    # [B, n, H]
        mask = anc[:, i, :, None]
        u[:, i] = beta[:, i, :, None] * (v[:, i] - first[:, :, 0] - ((ki * mask)[..., None] * u).sum(1))
        o[:, i] = scale * (first[:, :, 1] + ((qi * (mask | own_node[i][:, None]))[..., None] * u).sum(1))
    out_o, out_u = torch.empty_like(s["o"]), torch.empty_like(s["u"])
    out_o[rows[real]], out_u[rows[real]] = o[real].to(out_o.dtype), u[real]
    return dict(o=out_o, u=out_u)


def _windows(x, pool, s):
    """The three inputs before each row's own, oldest first, [N, 3, C]: of its nearest
    ancestors, then of what its request carries."""
    n = s["nmax"]
    rows, real = _padded(s, n)
    strict = _bits(s["anc"][rows], n) & torch.tril(torch.ones(n, n, dtype=torch.bool, device=DEV), -1)
    depth = strict.sum(-1)                                                 # [B, n]
    slot = s["slots"].long()[:, None].expand(-1, n)
    taps = []
    for back in (3, 2, 1):
        # the ancestor that has back - 1 others above it in the node's word
        above = torch.flip(torch.cumsum(torch.flip(strict.long(), [-1]), -1), [-1])
        at = (strict & (above == back)).long().argmax(-1)
        mine = x[torch.gather(rows, 1, at)]
        carried = pool[slot, (3 - back + depth).clamp(max=2)]
        taps.append(torch.where((depth >= back)[..., None], mine, carried))
    w = torch.stack(taps, 2)                                               # [B, n, 3, C]
    out = torch.empty(x.shape[0], 3, x.shape[1], dtype=x.dtype, device=DEV)
    out[rows[real]] = w[real]
    return out


def _plain_conv(s):
    got = {}
    for z, name in enumerate("qkv"):
        x = s["x"][z]
        window = torch.cat([_windows(x, s["conv_pool"][:, z], s), x[:, None]], 1).float()
        a = (window * s["w"][z].t()[None]).sum(1)
        y = a / (1.0 + torch.exp(-a))
        if z < 2:
            h = y.view(x.shape[0], -1, 128)
            y = (h / torch.sqrt((h * h).sum(-1, keepdim=True) + 1e-6)).view_as(a)
        got[name] = y.to(torch.bfloat16)
    return got


def _plain_accept(s):
    n, last, ps = s["nmax"], s["last"].long(), s["case"]["page"]
    rows, real = _padded(s, n)
    some = last >= 0
    word = s["anc"][s["cu"][:-1].long() + last.clamp(min=0)]
    path = _bits(word, n) & (torch.arange(n, device=DEV)[None] <= last[:, None])
    path = (path | (torch.arange(n, device=DEV)[None] == last[:, None])) & some[:, None]   # [B, n]
    # the KDA state: the path's decays, and each node's product behind the decays after it
    g, k, u = s["g"][rows], s["k"][rows].float(), s["u"][rows]
    B, _, H, _ = g.shape
    after = torch.triu(torch.ones(n, n, dtype=torch.bool, device=DEV), 1).float()
    flat = g.reshape(B, n, -1)
    decay = torch.exp(torch.matmul(path[:, None].float(), flat).view(B, H, 128))
    behind = torch.exp(torch.matmul(path[:, None].float() * after[None], flat).view(B, n, H, 128))
    behind = behind * k * path[:, :, None, None]
    at = s["slots"].long()
    S = s["pool"][at].float()
    S = S * decay[..., None] + torch.matmul(behind.permute(0, 2, 3, 1), u.permute(0, 2, 1, 3))
    s["pool"][at[some]] = S[some].to(s["pool"].dtype)
    # the carried inputs of the convolution: the last three of what there was and the path's
    order = torch.argsort((~path).long(), dim=1, stable=True)              # the path's nodes first
    length = path.sum(1)
    for z in range(3):
        old, x = s["conv_pool"][at, z], s["x"][z]
        new = []
        for r in range(3):
            i = length + r - 3                                             # the path's i-th input, or a carried one
            mine = x[torch.gather(rows, 1, torch.gather(order, 1, i.clamp(min=0)[:, None]))[:, 0]]
            kept = old[torch.arange(B, device=DEV), (r + length).clamp(max=2)]
            new.append(torch.where((i >= 0)[:, None], mine, kept))
        s["conv_pool"][at, z] = torch.stack(new, 1)
    # the attention layer's cache: the path's keys and values move together behind the context
    counts = (s["cu"][1:] - s["cu"][:-1]).long()
    context = s["seq_lens"].long() - counts
    moved = torch.arange(n, device=DEV)[None] < length[:, None]
    to, frm = context[:, None] + torch.arange(n, device=DEV)[None], context[:, None] + order

    def place(pos):
        pos = torch.where(moved, pos, torch.zeros_like(pos))
        return torch.gather(s["table"].long(), 1, pos // ps)[moved], (pos % ps)[moved]

    for cache in (s["k_cache"], s["v_cache"]):
        x = _raw(cache)[place(frm)]
        _raw(cache)[place(to)] = x
    return dict(pool=s["pool"], conv_pool=s["conv_pool"], k_cache=s["k_cache"], v_cache=s["v_cache"],
                kept=(context + length).int())


def _plain_pages(s):
    ps, table, shares = s["case"]["page"], s["table"], s["shares"]
    src, dst = s["src"].long(), s["dst"].long()
    n = s["seq_lens"].long()[src]
    full, part = n // ps, n % ps
    takes = (part > 0).long()
    off = torch.cumsum(takes, 0) - takes
    col = torch.arange(table.shape[1], device=DEV)[None]
    rows = table[src]
    ours = s["free"][off.clamp(max=s["free"].numel() - 1)]
    new = torch.where(col < full[:, None], rows, table[dst])
    new = torch.where((col == full[:, None]) & (part > 0)[:, None], ours[:, None], new)
    shared = rows[col.expand_as(rows) < full[:, None]].long()
    shares = shares + torch.bincount(shared, minlength=shares.numel()).int()
    from_page = torch.gather(rows, 1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    copies = torch.where((part > 0)[:, None], torch.stack([from_page, ours, part.int()], 1),
                         torch.tensor([-1, -1, 0], dtype=torch.int32, device=DEV)[None])
    table[dst] = new
    s["seq_lens"][dst] = n.int()
    # what the copied pages hold
    one = torch.arange(ps, device=DEV)[None].expand(copies.shape[0], ps)
    held = one < copies[:, 2:]
    for cache in (s["k_cache"], s["v_cache"]):
        raw = _raw(cache)
        raw[copies[:, 1:2].long().expand_as(one)[held], one[held]] = \
            raw[copies[:, :1].long().expand_as(one)[held], one[held]]
    # pages behind the kept lengths: one holder less, or free
    lo, hi = (s["kept"].long() + ps - 1) // ps, (s["seq_lens"].long() + ps - 1) // ps
    gone = table[(col >= lo[:, None]) & (col < hi[:, None])].long()
    times = torch.bincount(gone, minlength=shares.numel()).int()
    free = times > shares
    s["shares"].copy_(torch.where(free, torch.zeros_like(shares), shares - times))
    pages = torch.nonzero(free)[:, 0].int()
    s["freed"][:pages.numel()] = pages
    return dict(table=table, seq_lens=s["seq_lens"], shares=s["shares"], copies=copies,
                used=takes.sum()[None].int(), freed=s["freed"], num_freed=free.sum()[None].int(),
                k_cache=s["k_cache"], v_cache=s["v_cache"])


# --- what a pass cannot do without ---------------------------------------------------------

def work(case):
    op = case["op"]
    size = 1 if case.get("cache") == "fp8" else 2
    if op == "pages":
        ps, row = case["page"], 2 * case["Hkv"] * case["D"] * size
        src, dst, lens, grown, kept = _ends(case)
        shared = sum(lens[x] // ps for x in src)
        copied = sum(lens[x] % ps for x in src)
        gone = sum(_pages(n, ps) - _pages(m, ps) for n, m in zip(grown, kept))
        # table entries read and written, shares of the pages that are shared or left, lists, rows copied
        return dict(bytes=4 * (4 * shared + 4 * gone + 8 * len(src) + 2 * case["B"]) + 2 * copied * row, flops=0)
    counts = [len(t) for t in _trees(case)]
    N, B = sum(counts), case["B"]
    tree = 8 * N + 4 * B
    if op == "attend":
        Hq, keys = case["Hkv"] * case["G"], _lens(case)
        table = sum(_pages(n, case["page"]) for n in keys)
        return dict(bytes=2 * sum(keys) * case["Hkv"] * case["D"] * size + N * Hq * (4 * case["D"] + 4)
                    + 4 * (B + table) + tree,
                    flops=sum(4 * n * L * Hq * case["D"] for n, L in zip(counts, keys)))
    H = case["H"]
    if op == "conv":
        return dict(bytes=3 * H * 128 * (4 * N + 6 * B + 16) + tree, flops=3 * H * 128 * N * 12)
    state = 16384 * (4 if case["state"] == "fp32" else 2)
    if op == "recur":
        out = 4 if case["out"] == "fp32" else 2
        pairs = sum(bin(w).count("1") for t in _trees(case) for w in _words(t))
        return dict(bytes=B * H * state + N * H * (128 * (3 * 2 + 4 + out + 4) + 4) + tree,
                    flops=H * (N * 4 * 16384 + pairs * 8 * 128))
    # accept: states read and written, the paths' keys, decays and updates, the windows, the moved rows
    paths = [bin(_words(t)[e]).count("1") if e >= 0 else 0 for t, e in zip(_trees(case), _last(case))]
    moved = sum(2 * bin(_words(t)[e] & ~((1 << p) - 1)).count("1") if e >= 0 else 0
                for t, e, p in zip(_trees(case), _last(case), paths))
    some = sum(1 for p in paths if p > 0)
    return dict(bytes=some * H * 2 * state + sum(paths) * H * 128 * (2 + 4 + 4) + some * 2 * 9 * H * 128 * 2
                + moved * 2 * case["Hkv"] * case["D"] * size + 8 * B + tree,
                flops=H * 16384 * (some + 2 * sum(paths)))


# --- the definition in 64 bits -------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers and copies
    s = prepare(case, seed)
    return {"attend": _exact_attend, "recur": _exact_recur, "conv": _exact_conv,
            "accept": _exact_accept}[case["op"]](case, s)


def _exact_attend(case, s):
    Hkv, G, D, ps = case["Hkv"], case["G"], case["D"], case["page"]
    trees, lens = _trees(case), _lens(case)
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    ones = torch.ones(Hkv, device=DEV)
    ks = (ones if s["k_scale"] is None else s["k_scale"]).double()
    vs = (ones if s["v_scale"] is None else s["v_scale"]).double()
    row = 0
    for b, (tree, L) in enumerate(zip(trees, lens)):
        pages = s["table"][b, :_pages(L, ps)].long()
        k = _raw(s["k_cache"])[pages].view(s["k_cache"].dtype).flatten(0, 1)[:L].double() * ks[:, None]
        v = _raw(s["v_cache"])[pages].view(s["v_cache"].dtype).flatten(0, 1)[:L].double() * vs[:, None]
        for i in range(len(tree)):
            node, seen = i, list(range(L - len(tree)))
            drafts = []
            while node >= 0:
                drafts.append(L - len(tree) + node)
                node = tree[node]
            at = torch.tensor(seen + drafts[::-1], device=DEV)
            x = torch.einsum("hgd,nhd->hgn", s["q"][row].double().view(Hkv, G, D), k[at]) * s["scale"]
            lse[row] = torch.logsumexp(x, -1).view(-1)
            o[row] = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), v[at]).reshape(Hkv * G, D)
            row += 1
    return dict(o=o, lse=lse)


def _exact_recur(case, s):
    """The recurrence itself, a state for every node."""
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=DEV)
    u = torch.zeros_like(o)
    row = 0
    for b, tree in enumerate(_trees(case)):
        states, first = [], s["pool"][s["slots"][b].long()].double()
        for parent in tree:
            k, q, v = (s[x][row].double() for x in ("k", "q", "v"))
            S = torch.exp(s["g"][row].double())[:, :, None] * (first if parent < 0 else states[parent])
            u[row] = s["beta"][row].double()[:, None] * (v - torch.einsum("hkv,hk->hv", S, k))
            S = S + k[:, :, None] * u[row][:, None, :]
            o[row] = torch.einsum("hkv,hk->hv", S, s["scale"] * q)
            states.append(S)
            row += 1
    return dict(o=o, u=u)


def _path(tree, node):
    path = []
    while node >= 0:
        path.append(node)
        node = tree[node]
    return path[::-1]


def _exact_conv(case, s):
    got = {}
    for z, name in enumerate("qkv"):
        x, w = s["x"][z].double(), s["w"][z].double()
        y, row = torch.zeros_like(x), 0
        for b, tree in enumerate(_trees(case)):
            carried = s["conv_pool"][s["slots"][b].long(), z].double()
            for i in range(len(tree)):
                inputs = torch.cat([carried, x[[row + j for j in _path(tree, i)]]])[-4:]
                y[row + i] = (inputs * w.t()).sum(0)
            row += len(tree)
        y = y * torch.sigmoid(y)
        if z < 2:
            h = y.view(x.shape[0], -1, 128)
            y = (h * torch.rsqrt(h.square().sum(-1, keepdim=True) + 1e-6)).flatten(1)
        got[name] = y
    return got


def _exact_accept(case, s):
    trees, last = _trees(case), _last(case)
    pool, conv = s["pool"].double(), s["conv_pool"].double()
    caches = {x: s[x].double() for x in ("k_cache", "v_cache")}
    row = 0
    for b, tree in enumerate(trees):
        path, at = _path(tree, last[b]), int(s["slots"][b])
        for j in path:
            pool[at] = pool[at] * torch.exp(s["g"][row + j].double())[:, :, None] \
                + s["k"][row + j].double()[:, :, None] * s["u"][row + j].double()[:, None, :]
        for z in range(3):
            conv[at, z] = torch.cat([conv[at, z], s["x"][z][[row + j for j in path]].double()])[-3:]
        context = _lens(case)[b] - len(tree)
        table = s["table"][b].tolist()
        for r, j in enumerate(path):
            (tp, to), (fp, fo) = (divmod(context + i, case["page"]) for i in (r, j))
            for x in caches.values():
                x[table[tp], to] = x[table[fp], fo]
        row += len(tree)
    return dict(pool=pool, conv_pool=conv, kept=None, **caches)
