"""The paged key-value cache operators as measured cases: each in its plain form
(elementary torch operations in 32 bits) and as the calls a user makes.

A serving step of the softmax-attention layers that sit between KDA layers runs
the three in this order: ``plan`` (block table and slot map of the step, once
for all layers), ``append`` (the step's new keys and values into the cache) and
``decode`` (one new token per sequence attends over its cached keys).
"""
import math
import random

import torch

own = False

DEV = "cuda"
FP8_MAX = 448.0


# --- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # eight requests decoding: the smallest call of a serving loop, pure latency
        dict(name="plan_decode_b8", op="plan", B=8, page=16, cached_hi=900, new_lo=1, new_hi=1, mix=7),
        # a mixed step: mostly decoding requests, some prompts being prefilled
        dict(name="plan_mixed_b256", op="plan", B=256, page=16, cached_hi=6000, new_lo=1, new_hi=401,
             mix=8),
        # many requests with whole prompts to place: the largest step (about 260 thousand tokens)
        dict(name="plan_prompts_b2048", op="plan", B=2048, page=64, cached_hi=3000, new_lo=1,
             new_hi=1025, mix=9),
        # one decode step of a small batch: 32 rows to write, latency
        dict(name="append_decode_n32", op="append", N=32, Hkv=8, D=128, page=16, cache="bf16",
             order="token", fused=True, mix=1),
        # a prefilled prompt of 16 thousand tokens, k and v slices of one fused projection
        dict(name="append_prompt_n16384", op="append", N=16384, Hkv=8, D=128, page=64, cache="bf16",
             order="token", fused=True, mix=2),
        # an odd number of tokens into an 8-bit cache with head-major pages
        dict(name="append_fp8_n9001", op="append", N=9001, Hkv=4, D=256, page=32, cache="fp8",
             order="head", fused=False, mix=3),
        # one short conversation: latency of a single-request decode
        dict(name="decode_b1_l77", op="decode", B=1, lo=77, hi=77, Hkv=8, G=4, D=128, page=16,
             cache="bf16", order="token", out="bf16", mix=1),
        # a small batch at 96 query heads (12 to a key head), odd ragged lengths and odd pages
        dict(name="decode_b9_g12", op="decode", B=9, lo=500, hi=3001, Hkv=8, G=12, D=128, page=24,
             cache="bf16", order="token", out="bf16", mix=2),
        # continuous batching: lengths over three decades, one to sixteen thousand
        dict(name="decode_b64_ragged", op="decode", B=64, lo=16, hi=16384, Hkv=8, G=8, D=128, page=64,
             cache="bf16", order="head", out="bf16", mix=3),
        # one request with a very long context: all of the split over the length
        dict(name="decode_b1_l262149", op="decode", B=1, lo=262149, hi=262149, Hkv=8, G=8, D=128,
             page=64, cache="bf16", order="token", out="bf16", mix=4),
        # a large batch over an 8-bit cache, the largest call
        dict(name="decode_b256_fp8", op="decode", B=256, lo=3500, hi=8192, Hkv=8, G=8, D=128, page=64,
             cache="fp8", order="head", out="bf16", mix=5),
        # one key head to each query head, 64 channels, fp32 outputs (joined with other partial results)
        dict(name="decode_b24_mha_d64", op="decode", B=24, lo=1000, hi=4097, Hkv=32, G=1, D=64, page=16,
             cache="bf16", order="token", out="fp32", mix=6),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "decode", "decode", "decode"])
    page = rng.choice([16, 16, 24, 32, 64, 64, 128])
    mix = rng.randrange(1 << 30)
    if op == "plan":
        B = _log_int(rng, 1, 2048)
        return dict(op=op, B=B, page=page, cached_hi=_log_int(rng, 1, 6000), new_lo=rng.choice([0, 1]),
                    new_hi=_log_int(rng, 1, max(1, min(4096, 262144 // B))), mix=mix)
    Hkv, D = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([64, 128, 128, 256])
    cache, order = rng.choice(["bf16", "bf16", "fp8"]), rng.choice(["token", "head"])
    if op == "append":
        most = 16384 * 8 * 128 // (Hkv * D)
        return dict(op=op, N=_log_int(rng, 1, most), Hkv=Hkv, D=D, page=page, cache=cache, order=order,
                    fused=rng.random() < 0.5, mix=mix)
    G = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24])
    most = 262144 * 8 * 128 // (Hkv * D)  # keys of all sequences together
    B = _log_int(rng, 1, 256)
    hi = _log_int(rng, 1, max(1, min(262144, most // B)))
    return dict(op=op, B=B, lo=max(0, hi // rng.choice([1, 2, 16, 1000]) - 1), hi=hi, Hkv=Hkv, G=G, D=D,
                page=page, cache=cache, order=order, out=rng.choice(["bf16", "bf16", "fp32"]), mix=mix)


def _lens(case):
    """The lengths of a case's requests: plain numbers of the case, the same for every seed."""
    rng = random.Random(case["mix"])
    if case["op"] == "plan":
        cached = [rng.choice([0, rng.randint(0, case["cached_hi"]), rng.randint(0, case["cached_hi"])])
                  for _ in range(case["B"])]
        # half of the requests decode (one token, or the least), the others prefill
        new = [case["new_lo"] if rng.random() < 0.5 else rng.randint(case["new_lo"], case["new_hi"])
               for _ in range(case["B"])]
        return cached, new
    lo, hi = case["lo"], case["hi"]
    if hi <= 8 * max(lo, 1):
        return [rng.randint(lo, hi) for _ in range(case["B"])]
    # spread over the lengths' logarithm; where the least is 0, some requests hold nothing yet
    return [0 if lo == 0 and rng.random() < 0.1 else _log_int(rng, max(lo, 1), hi)
            for _ in range(case["B"])]


def _pages(n, ps):
    return -(-n // ps)


# --- inputs --------------------------------------------------------------------------------

def _pool(num_pages, page, Hkv, D, cache, order, gen, sigma=None):
    """A cache [num_pages, page, Hkv, D] (a view where the pages are stored head by head)."""
    dtype = torch.float8_e4m3fn if cache == "fp8" else torch.bfloat16
    shape = (num_pages, Hkv, page, D) if order == "head" else (num_pages, page, Hkv, D)
    t = torch.zeros(shape, dtype=dtype, device=DEV)
    if sigma is not None:
        for i in range(0, num_pages, 4096):  # in parts: the fp32 draw of a whole pool would be large
            part = t[i:i + 4096]
            part.copy_((torch.randn(part.shape, device=DEV, generator=gen) * sigma))
    return t.permute(0, 2, 1, 3) if order == "head" else t


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 1000003 + case["mix"] % 99991)
    s = dict(case=case)
    ps = case["page"]
    i32 = dict(dtype=torch.int32, device=DEV)
    if case["op"] == "plan":
        cached, new = _lens(case)
        B, width = case["B"], max(_pages(c + n, ps) for c, n in zip(cached, new)) + 2
        held = [_pages(c, ps) for c in cached]
        needs = sum(_pages(c + n, ps) - h for c, n, h in zip(cached, new, held))
        num_pages = sum(held) + needs + 64
        order = torch.randperm(num_pages, device=DEV, generator=gen).to(torch.int32)
        h = torch.tensor(held, device=DEV)
        first = torch.cumsum(h, 0) - h
        col = torch.arange(width, device=DEV)[None]
        at = (first[:, None] + col).clamp(max=num_pages - 1)
        s["table"] = torch.where(col < h[:, None], order[at], torch.full_like(at, -1, dtype=torch.int32))
        s["table"] = s["table"].to(torch.int32).contiguous()
        s["free"] = order[sum(held):].contiguous()
        s["cached"], s["new"] = torch.tensor(cached, **i32), torch.tensor(new, **i32)
        N = sum(new) + 3  # a buffer with room for more tokens than this step has
        s["N"], s["num_pages"] = N, num_pages
        s["seq_lens"], s["cu"] = torch.empty(B, **i32), torch.empty(B + 1, **i32)
        s["slots"], s["used"] = torch.empty(N, **i32), torch.empty(1, **i32)
        return s
    Hkv, D = case["Hkv"], case["D"]
    fp8 = case["cache"] == "fp8"
    s["k_scale"] = s["v_scale"] = None
    if fp8:  # a head's scale puts its largest values near the top of the 8-bit range
        s["k_scale"] = 0.01 + 0.02 * torch.rand(Hkv, device=DEV, generator=gen)
        s["v_scale"] = 0.01 + 0.02 * torch.rand(Hkv, device=DEV, generator=gen)
    if case["op"] == "append":
        N = case["N"]
        num_pages = _pages(N, ps) + 7
        s["slots"] = torch.randperm(num_pages * ps, device=DEV, generator=gen)[:N].to(torch.int32)
        if N > 4:  # runs of a page's slots in order, as requests have them, and one token left out
            runs = torch.randperm(num_pages, device=DEV, generator=gen).to(torch.int64)
            run = (runs[:, None] * ps + torch.arange(ps, device=DEV)[None]).reshape(-1)[:N]
            s["slots"] = run.to(torch.int32)
            s["slots"][N // 2] = -1
        if case["fused"]:  # [q | k | v] rows of one projection; q is as wide as two kv streams here
            rows = torch.randn(N, 4 * Hkv * D, device=DEV, generator=gen).to(torch.bfloat16)
            s["k"] = rows[:, 2 * Hkv * D:3 * Hkv * D].view(N, Hkv, D)
            s["v"] = rows[:, 3 * Hkv * D:].view(N, Hkv, D)
        else:
            s["k"] = torch.randn(N, Hkv, D, device=DEV, generator=gen).to(torch.bfloat16)
            s["v"] = torch.randn(N, Hkv, D, device=DEV, generator=gen).to(torch.bfloat16)
        s["k_cache"] = _pool(num_pages, ps, Hkv, D, case["cache"], case["order"], gen)
        s["v_cache"] = _pool(num_pages, ps, Hkv, D, case["cache"], case["order"], gen)
        if own:
            import gated_delta_rule_33_gb300 as kda
            s["cache"] = kda.PagedCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        return s
    lens = _lens(case)
    B, Hq = case["B"], case["Hkv"] * case["G"]
    width = max(1, max(_pages(n, ps) for n in lens))
    held = torch.tensor([_pages(n, ps) for n in lens], device=DEV)
    num_pages = int(held.sum()) + 5
    order = torch.randperm(num_pages, device=DEV, generator=gen).to(torch.int32)
    first = torch.cumsum(held, 0) - held
    at = (first[:, None] + torch.arange(width, device=DEV)[None]).clamp(max=num_pages - 1)
    s["table"] = order[at].contiguous()
    s["seq_lens"] = torch.tensor(lens, **i32)
    # scores of spread about 2: some keys matter much more than others
    s["q"] = (2.0 * torch.randn(B, Hq, D, device=DEV, generator=gen)).to(torch.bfloat16)
    s["k_cache"] = _pool(num_pages, ps, Hkv, D, case["cache"], case["order"], gen, 50.0 if fp8 else 1.0)
    s["v_cache"] = _pool(num_pages, ps, Hkv, D, case["cache"], case["order"], gen, 50.0 if fp8 else 1.0)
    s["scale"] = D ** -0.5
    s["o"] = torch.empty(B, Hq, D, device=DEV,
                         dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16)
    s["lse"] = torch.empty(B, Hq, device=DEV)
    if own:
        import gated_delta_rule_33_gb300 as kda
        s["cache"] = kda.PagedCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        s["ws"] = torch.empty(max(16, kda.kda_paged_decode_workspace_size(B, Hq, Hkv, D)),
                              dtype=torch.uint8, device=DEV)
    return s


# --- one pass ------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        import gated_delta_rule_33_gb300 as kda
        if op == "plan":
            kda.kda_page_plan(s["cached"], s["new"], s["free"], s["table"], s["case"]["page"],
                              s["num_pages"], s["seq_lens"], s["cu"], s["slots"], s["used"])
            return dict(table=s["table"], seq_lens=s["seq_lens"], cu=s["cu"], slots=s["slots"],
                        used=s["used"])
        if op == "append":
            kda.kda_paged_append(s["k"], s["v"], s["slots"], s["cache"])
            return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
        kda.kda_paged_decode(s["q"], s["cache"], s["table"], s["seq_lens"], s["scale"], s["o"],
                             s["lse"], s["ws"])
        return dict(o=s["o"], lse=s["lse"])
    return {"plan": _plain_plan, "append": _plain_append, "decode": _plain_decode}[op](s)


def _plain_plan(s):
    ps, cached, new, table = s["case"]["page"], s["cached"].long(), s["new"].long(), s["table"]
    total = cached + new
    held = (cached + ps - 1) // ps
    need = (total + ps - 1) // ps - held
    end = torch.cumsum(need, 0)
    col = torch.arange(table.shape[1], device=DEV)[None]
    take = (end - need)[:, None] + col - held[:, None]
    mine = (col >= held[:, None]) & (col < (held + need)[:, None])
    table = torch.where(mine, s["free"][take.clamp(0, s["free"].numel() - 1)], table)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(new, 0)])
    t = torch.arange(s["N"], device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=cached.numel() - 1)
    pos = cached[b] + t - cu[b]
    page = table[b, (pos // ps).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(t < cu[-1], page * ps + pos % ps, torch.full_like(t, -1))
    return dict(table=table, seq_lens=total.int(), cu=cu.int(), slots=slots.int(), used=end[-1:].int())


def _plain_append(s):
    ps, kept = s["case"]["page"], s["slots"] >= 0
    at = s["slots"][kept].long()
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        x = x[kept].float()
        if scale is not None:
            x = (x / scale[:, None]).clamp(-FP8_MAX, FP8_MAX)
        x, raw = x.to(cache.dtype), torch.uint8 if scale is not None else cache.dtype
        cache.view(raw)[at // ps, at % ps] = x.view(raw)
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])


def _gather(cache, scale, table, length):
    """The first `length` keys of every request, [B, Hkv, length, D] in 32 bits."""
    x = cache.view(torch.uint8)[table.long()].view(cache.dtype) if cache.element_size() == 1 \
        else cache[table.long()]
    x = x.flatten(1, 2)[:, :length].permute(0, 2, 1, 3).float()
    return x if scale is None else x * scale[None, :, None, None]


def _plain_decode(s):
    c = s["case"]
    B, Hkv, G, D = c["B"], c["Hkv"], c["G"], c["D"]
    length = s["table"].shape[1] * c["page"]
    q = s["q"].float().view(B, Hkv, G, D) * s["scale"]
    scores = torch.matmul(q, _gather(s["k_cache"], s["k_scale"], s["table"], length).transpose(2, 3))
    seen = torch.arange(length, device=DEV)[None] < s["seq_lens"][:, None]
    scores = torch.where(seen[:, None, None], scores, torch.full_like(scores, -math.inf))
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(scores - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _gather(s["v_cache"], s["v_scale"], s["table"], length))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return dict(o=o.view(B, Hkv * G, D).to(s["o"].dtype), lse=(m + torch.log(total)).view(B, Hkv * G))


# --- what a pass cannot do without ---------------------------------------------------------

def work(case):
    ps = case["page"]
    if case["op"] == "plan":
        cached, new = _lens(case)
        need = sum(_pages(c + n, ps) - _pages(c, ps) for c, n in zip(cached, new))
        B, N = case["B"], sum(new) + 3
        # lengths in, lengths and offsets out, pages taken from the free list into the table, slots out
        return dict(bytes=4 * (2 * B + B + B + 1 + 2 * need + N + 1), flops=0)
    Hkv, D, size = case["Hkv"], case["D"], 1 if case["cache"] == "fp8" else 2
    if case["op"] == "append":
        N = case["N"]
        return dict(bytes=4 * N + 2 * N * Hkv * D * (2 + size), flops=0)
    keys, B, Hq = sum(_lens(case)), case["B"], Hkv * case["G"]
    out = 4 if case["out"] == "fp32" else 2
    table = sum(_pages(n, ps) for n in _lens(case))
    return dict(bytes=2 * keys * Hkv * D * size + B * Hq * (D * (2 + out) + 4) + 4 * (B + table),
                flops=4 * keys * Hq * D)


# --- the definition in 64 bits -------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    ps = case["page"]
    if case["op"] == "append":
        got = {}
        for name, cache, scale in (("k", s["k_cache"], s["k_scale"]), ("v", s["v_cache"], s["v_scale"])):
            flat = torch.zeros(cache.shape[0] * ps, case["Hkv"], case["D"], dtype=torch.float64, device=DEV)
            for part in torch.nonzero(s["slots"] >= 0).flatten().split(65536):
                x = s[name][part].double()
                if scale is not None:  # four significant bits, steps of 2^-9 at the least, 448 at most
                    x = x / scale.double()[:, None]
                    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
                    x = (torch.round(x / step) * step).clamp(-FP8_MAX, FP8_MAX)
                flat[s["slots"][part].long()] = x
            got[name + "_cache"] = flat.view(cache.shape)
        return got
    lens = _lens(case)
    B, Hkv, G, D = case["B"], case["Hkv"], case["G"], case["D"]
    o = torch.zeros(B, Hkv * G, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hkv * G), -math.inf, dtype=torch.float64, device=DEV)
    ones = torch.ones(Hkv, device=DEV)
    ks = (ones if s["k_scale"] is None else s["k_scale"]).double()
    vs = (ones if s["v_scale"] is None else s["v_scale"]).double()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pages = s["table"][b, :_pages(n, ps)].tolist()
        k = torch.cat([s["k_cache"][p].double() for p in pages])[:n] * ks[:, None]
        v = torch.cat([s["v_cache"][p].double() for p in pages])[:n] * vs[:, None]
        x = torch.einsum("hgd,nhd->hgn", s["q"][b].double().view(Hkv, G, D), k) * s["scale"]
        lse[b] = torch.logsumexp(x, -1).view(-1)
        o[b] = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), v).reshape(Hkv * G, D)
    return dict(o=o, lse=lse)
