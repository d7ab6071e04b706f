"""What the operators of the paged caches are measured on: the cases, their inputs, and the operators' plain forms.

attention  one softmax over a bf16 window and the entries of a cache held in 8 bits (e4m3, a power-of-two scale for each block
           of entries) in pages, with a sink per head and the inverse rotation of the last 64 dims: over selected entries
           (list) or over every visible one (range)
append     entries of a segment quantised into the pages (a block's scale grows with its rows), then read back as bf16
fork       slots kept, forked and freed by a parent map, pages reserved for what comes next
compact    live pages moved to the front of their pools
indexer    sum_h w_h ReLU(q_h . k_s) over bf16 index rows in pages
"""

import math

import torch

own = False

D, ROPE, BASE = 512, 64, 10000.0
E4M3_MAX = 448.0


def listed():
    return [
        # the layer's headline configuration: 64 requests at 32K, 1024 of 8192 entries each
        dict(name="attention, 64 at 32K", kind="attention", B=64, S=1, H=128, ctx=32768, ratio=4, topk=1024, window=128, page=64, block=16),
        # a segment of a prefill, the window rows of the segment in the ring
        dict(name="attention, segment of 2000", kind="attention", B=1, S=2000, H=128, ctx=9001, ratio=4, topk=1024, window=128, page=64, block=16),
        # one request's HCA decode step early in a conversation; latency counts
        dict(name="attention, one request, every entry", kind="attention", B=1, S=1, H=128, ctx=5000, ratio=128, topk=0, window=128, page=64, block=16),
        # HCA decode: every entry of ratio 128, here with contexts of 200K and pages of an odd fill
        dict(name="attention, 24 at 200K, every entry", kind="attention", B=24, S=1, H=128, ctx=200003, ratio=128, topk=0, window=128, page=32, block=1),
        # the decode step of 64 requests whose token completes a group: one entry each joins a block with earlier rows
        dict(name="append, one entry each", kind="append", B=64, S=1, ctx=32763, ratio=4, page=64, block=16),
        # the entries of an 8K prefill chunk of four requests, behind 1001 tokens
        dict(name="append, 8K prefill", kind="append", B=4, S=8192, ctx=1001, ratio=4, page=64, block=16),
        # two samples of one short prompt
        dict(name="fork, two of four", kind="fork", slots=4, groups=2, entries=300, page=64, block=16, pools=2),
        # 16 prompts of up to 32K, four samples each, main and index pages of one table
        dict(name="fork, 16 prompts by four", kind="fork", slots=64, groups=16, entries=8100, page=64, block=16, pools=2),
        # a small pool after one request of four left
        dict(name="compact, a small pool", kind="compact", slots=4, pages=256, live=0.7, page=64, block=16),
        # a pool of 16K pages of which about half are live, after requests left
        dict(name="compact, half of 16K pages", kind="compact", slots=64, pages=16384, live=0.5, page=64, block=16),
        # index scores of a few tokens of one request over 3001 tokens of context
        dict(name="indexer, five tokens", kind="indexer", B=1, S=5, HI=64, ctx=3001, ratio=4, page=64),
        # the headline decode configuration's index scan, in pages
        dict(name="indexer, 64 at 32K", kind="indexer", B=64, S=1, HI=64, ctx=32768, ratio=4, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "attention", "append", "fork", "compact", "indexer"])
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (1, 2, 4, 8, 16, 32, 64) if b <= page])
    if kind == "attention":
        H, window = rng.choice([8, 64, 100, 128, 128]), rng.choice([16, 100, 128, 128, 200])
        ratio, topk = rng.choice([(4, 1024), (4, rng.randint(1, 2048)), (128, 0)])
        if rng.random() < 0.3:  # a segment
            B, S = 1, _log(rng, 2, 1000)
            ctx = S + _log(rng, 1, 8000)
        else:
            B, S = _log(rng, 1, 64), 1
            ctx = _log(rng, 4, 1048576 if B <= 8 else 65536)
        return dict(kind=kind, B=B, S=S, H=H, ctx=ctx, ratio=ratio, topk=topk, window=window, page=page, block=block)
    if kind == "append":
        B, ratio = _log(rng, 1, 64), rng.choice([4, 4, 128])
        S = 1 if rng.random() < 0.4 else _log(rng, ratio, max(ratio + 1, 32768 // B))
        return dict(kind=kind, B=B, S=S, ctx=_log(rng, 4, 32768), ratio=ratio, page=page, block=block)
    if kind == "fork":
        slots = _log(rng, 2, 64)
        return dict(kind=kind, slots=slots, groups=rng.randint(1, slots), entries=_log(rng, 1, 8000), page=page, block=block, pools=rng.choice([1, 2]))
    if kind == "compact":
        pages = _log(rng, 16, 8192)
        return dict(kind=kind, slots=_log(rng, 1, min(64, pages)), pages=pages, live=round(rng.uniform(0.05, 0.95), 3), page=page, block=block)
    B = _log(rng, 1, 64)
    S = 1 if B > 1 else _log(rng, 1, 300)
    return dict(kind="indexer", B=B, S=S, HI=rng.choice([8, 32, 64, 128]), ctx=S + _log(rng, 8, 32768), ratio=4, page=page)


# ------------------------------------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _pow2_scale(amax):
    """The least power of two 2^k, k >= -100, with amax <= 448 * 2^k."""
    frac, ex = torch.frexp(amax / E4M3_MAX)
    k = torch.where(frac == 0.5, ex - 1, ex)
    k = torch.where(amax == 0, torch.full_like(k, -100), k).clamp(min=-100)
    return ((k + 127) << 23).view(torch.float32)  # by its bits: ldexp goes through pow, which is inexact on the GPU


def _filled_pages(g, pages, page, block):
    """Pages of rows as the compressor leaves them (each of unit RMS), quantised block by block."""
    x = _randn(g, pages, page // block, block * D)
    s = _pow2_scale(x.abs().amax(-1))
    return (x / s[..., None]).to(torch.float8_e4m3fn).view(pages, page, D), s


def _table(g, slots, max_pages, pages, used):
    """Each slot's pages in random places of the pool; slot b maps the first used[b] of its pages."""
    perm = torch.randperm(pages, generator=g, device="cuda")[: slots * max_pages].to(torch.int32).view(slots, max_pages)
    lp = torch.arange(max_pages, device="cuda")
    return torch.where(lp[None, :] < used[:, None], perm, torch.full_like(perm, -1)).contiguous()


def _refs(table, pages):
    t = table[table >= 0].long()
    return torch.bincount(t, minlength=pages).to(torch.int32)


def _handles(s, names):
    """The framework's page table and caches over the state's tensors, as a user's program keeps them."""
    from long_context_decode_c4a_b200 import ops

    s["ops"] = ops
    s["book"] = ops.PageTable(s["table"], s["refs"], s["case"]["page"])
    s["caches"] = [ops.PagedCache(s["book"], s[p], s[sc] if sc else None) for p, sc in names]
    return ops


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    kind, page = case["kind"], case["page"]
    if kind == "attention":
        B, S, H, W, ratio, ctx, K = case["B"], case["S"], case["H"], case["window"], case["ratio"], case["ctx"], case["topk"]
        # requests end at different places of the last eighth before ctx; a segment's tokens follow one another
        last = ctx - 1 - torch.randint(0, max(1, (ctx - S) // 8 + 1), (B,), generator=g, device="cuda")
        last[0] = ctx - 1
        q_pos = (last[:, None] - S + 1 + torch.arange(S, device="cuda")[None, :]).to(torch.int32)
        max_entries = max(1, ctx // ratio)
        max_pages = -(-max_entries // page)
        pool = B * max_pages
        s["pages"], s["scales"] = _filled_pages(g, pool, page, case["block"])
        s["table"] = _table(g, B, max_pages, pool, -(-((last + 1) // ratio) // page))
        s["refs"] = _refs(s["table"], pool)
        q = _randn(g, B, S, H, D)
        s["q"] = (q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)
        cap = W if S == 1 else S + W
        s["ring"] = _randn(g, B, cap, D, dtype=torch.bfloat16)
        s["sink"] = _randn(g, H)
        s["q_pos"] = q_pos.contiguous()
        s["topk"] = None
        if K:
            vis = (q_pos.long() + 1) // ratio
            r = torch.rand(B, S, max_entries, generator=g, device="cuda")
            r = r.masked_fill(torch.arange(max_entries, device="cuda") >= vis[..., None], -1.0)
            v, i = r.topk(min(K, max_entries), dim=-1)
            i = torch.where(v >= 0, i, torch.full_like(i, max_entries)).sort(-1).values
            i = torch.where(i < max_entries, i, torch.full_like(i, -1)).to(torch.int32)
            s["topk"] = torch.nn.functional.pad(i, (0, K - i.shape[-1]), value=-1).contiguous()
        if own:
            ops = _handles(s, [("pages", "scales")])
            s["out"] = torch.empty_like(s["q"])
            s["ws"] = ops.workspace(ops._lib.CSA_WS_SPARSE_ATTN, B, S, 1, 1)
    elif kind == "append":
        B, S, ratio, ctx, block = case["B"], case["S"], case["ratio"], case["ctx"], case["block"]
        # decode: every request's token completes a group; a segment starts anywhere near ctx
        back = torch.randint(0, max(1, ctx // 8), (B,), generator=g, device="cuda")
        start = (ctx - back) // ratio * ratio + ratio - 1 if S == 1 else ctx - back
        s["start"] = start.to(torch.int32)
        cap = (ctx + ratio + S) // ratio + 1
        max_pages = -(-cap // page)
        pool = B * max_pages
        s["pages"], s["scales"] = _filled_pages(g, pool, page, block)
        s["table"] = _table(g, B, max_pages, pool, torch.full((B,), max_pages, device="cuda"))
        s["refs"] = _refs(s["table"], pool)
        # new rows: unit RMS, here and there a row four times as large
        big = torch.where(torch.rand(B, cap, 1, generator=g, device="cuda") < 0.1, 4.0, 1.0)
        s["rows"] = (_randn(g, B, cap, D) * big).to(torch.bfloat16)
        n = S // ratio + 2
        first = start // ratio // block * block  # read back from the start of the first block that the append touches
        idx = first[:, None] + torch.arange(n + block - 1, device="cuda")[None, :]
        idx = torch.where(idx < ((start + S) // ratio)[:, None], idx, torch.full_like(idx, -1))
        s["idx"] = idx.to(torch.int32).contiguous()
        s["out"] = torch.zeros(B, idx.shape[1], D, dtype=torch.bfloat16, device="cuda")
        if own:
            _handles(s, [("pages", "scales")])
    elif kind == "fork":
        R, G, E = case["slots"], case["groups"], case["entries"]
        max_pages = -(-(E + 1) // page) + 1
        pool = R * max_pages
        entries = E - torch.randint(0, max(1, E // 4), (R,), generator=g, device="cuda")
        kept = torch.arange(R, device="cuda") < G
        # the first G slots hold the prompts; the rest are empty, but for one that holds an old request
        old = torch.where(kept | (torch.arange(R, device="cuda") == R - 1), entries, torch.zeros_like(entries))
        s["table"] = _table(g, R, max_pages, pool, -(-old // page))
        s["refs"] = _refs(s["table"], pool)
        s["parent"] = (torch.arange(R, device="cuda") % G).to(torch.int32)
        s["entries"] = old.to(torch.int32)
        s["after"] = (old[s["parent"].long()] + 1).to(torch.int32)
        s["pages"], s["scales"] = _filled_pages(g, pool, page, case["block"])
        if case["pools"] == 2:
            s["index"] = _randn(g, pool, page, 128, dtype=torch.bfloat16)
        if own:
            _handles(s, [("pages", "scales")] + ([("index", None)] if case["pools"] == 2 else []))
    elif kind == "compact":
        R, P = case["slots"], case["pages"]
        max_pages = max(1, P // R)
        used = (torch.rand(R, generator=g, device="cuda") * 2 * case["live"] * max_pages).long().clamp(0, max_pages)
        s["table0"] = _table(g, R, max_pages, P, used)
        s["refs0"] = _refs(s["table0"], P)
        s["table"], s["refs"] = s["table0"].clone(), s["refs0"].clone()
        s["pages"], s["scales"] = _filled_pages(g, P, page, case["block"])
        s["map"] = torch.empty(P, dtype=torch.int32, device="cuda")
        s["live"] = torch.empty(1, dtype=torch.int32, device="cuda")
        if own:
            _handles(s, [("pages", "scales")])
    else:
        B, S, HI, ctx, ratio = case["B"], case["S"], case["HI"], case["ctx"], case["ratio"]
        last = ctx - 1 - torch.randint(0, max(1, (ctx - S) // 8 + 1), (B,), generator=g, device="cuda")
        s["q_pos"] = (last[:, None] - S + 1 + torch.arange(S, device="cuda")[None, :]).to(torch.int32).contiguous()
        max_pages = -(-max(1, ctx // ratio) // page)
        pool = B * max_pages
        s["index"] = _randn(g, pool, page, 128, dtype=torch.bfloat16)
        s["table"] = _table(g, B, max_pages, pool, -(-((last + 1) // ratio) // page))
        s["refs"] = _refs(s["table"], pool)
        s["q"] = _randn(g, B, S, HI, 128, dtype=torch.bfloat16)
        s["w"] = _randn(g, B, S, HI) / math.sqrt(128) / math.sqrt(HI)
        s["scores"] = torch.zeros(B, S, max_pages * page, device="cuda")
        if own:
            ops = _handles(s, [("index", None)])
            s["ws"] = ops.workspace(ops._lib.CSA_WS_SPARSE_ATTN, B, S, 1, 1)
    return s


# ------------------------------------------------------------------------------------------------ one pass


def run(s):
    return {"attention": _attention, "append": _append, "fork": _fork, "compact": _compact, "indexer": _indexer}[s["case"]["kind"]](s)


def _candidates(s, dtype):
    """Rows [B*S, W + K, D] of every query's candidates and which of them count."""
    c, t = s["case"], s["q_pos"].long()
    B, S = t.shape
    cap, page = s["ring"].shape[1], c["page"]
    p = t[..., None] - torch.arange(c["window"] - 1, -1, -1, device=t.device)
    b = torch.arange(B, device=t.device)[:, None, None]
    win = s["ring"][b, p.clamp(min=0) % cap].to(dtype)
    if s["topk"] is not None:
        e = s["topk"].long()
    else:
        e = torch.arange(s["table"].shape[1] * page, device=t.device).expand(B, S, -1)
        e = torch.where(e < ((t + 1) // c["ratio"])[..., None], e, torch.full_like(e, -1))
    row = s["table"].long()[b, e.clamp(min=0) // page].clamp(min=0) * page + e.clamp(min=0) % page
    ent = s["pages"].view(-1, D)[row].to(dtype) * s["scales"].view(-1)[row // c["block"]].to(dtype)[..., None]
    ok = torch.cat([p >= 0, e >= 0], -1)
    rows = torch.cat([win, ent], 2) * ok[..., None].to(dtype)
    return rows.view(B * S, -1, D), ok.view(B * S, -1)


def _attention(s):
    c = s["case"]
    if own:
        if s["topk"] is not None:
            return s["ops"].sparse_attn8(s["q_pos"], s["q"], s["ring"], s["caches"][0], s["topk"], s["sink"], c["window"], ratio=c["ratio"], out=s["out"], ws=s["ws"])
        return s["ops"].hca_attn8(s["q_pos"], s["q"], s["ring"], s["caches"][0], s["sink"], c["window"], ratio=c["ratio"], out=s["out"], ws=s["ws"])
    rows, ok = _candidates(s, torch.float32)
    q = s["q"].float().view(rows.shape[0], c["H"], D)
    x = torch.matmul(q, rows.transpose(1, 2)).mul_(1 / math.sqrt(D)).masked_fill_(~ok[:, None, :], -math.inf)
    m = torch.maximum(x.amax(-1), s["sink"])
    p = x.sub_(m[..., None]).exp_()
    o = torch.matmul(p, rows) / (p.sum(-1) + torch.exp(s["sink"] - m))[..., None]
    ang = -s["q_pos"].double().view(-1, 1, 1) * BASE ** (-2.0 * torch.arange(ROPE // 2, device=o.device, dtype=torch.float64) / ROPE)
    cos, sin = ang.cos().float(), ang.sin().float()
    a, b = o[..., D - ROPE :: 2], o[..., D - ROPE + 1 :: 2]
    rot = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([o[..., : D - ROPE], rot], -1).to(torch.bfloat16).view(s["q"].shape)


def _append(s):
    c = s["case"]
    block, page, ratio, S = c["block"], c["page"], c["ratio"], c["S"]
    if own:
        s["ops"].cache_append(s["caches"][0], s["start"], S, s["rows"], ratio)
        return [s["ops"].cache_read(s["caches"][0], s["idx"], out=s["out"]), s["scales"]]
    dev, B = s["start"].device, s["start"].shape[0]
    e0, e1 = (s["start"].long() // ratio)[:, None, None], ((s["start"].long() + S) // ratio)[:, None, None]
    nb = (S // ratio + 1 + block - 1) // block + 1
    e = (e0 // block + torch.arange(nb, device=dev)[None, :, None]) * block + torch.arange(block, device=dev)
    new, old = (e >= e0) & (e < e1), (e < e0)
    b = torch.arange(B, device=dev)[:, None, None]
    row = s["table"].long()[b, (e // page).clamp(max=s["table"].shape[1] - 1)] * page + e % page
    blk = row[..., 0] // block
    pages, scales = s["pages"].view(-1, D), s["scales"].view(-1)
    x = s["rows"][b, e.clamp(max=s["rows"].shape[1] - 1)].float()
    need = _pow2_scale((x * new[..., None]).abs().amax((-1, -2)))
    had = torch.where(old.any(-1), scales[blk], torch.zeros_like(need))
    sc = torch.maximum(need, had)
    held = pages[row].float() * scales[blk][..., None, None]
    v = (torch.where(new[..., None], x, held) / sc[..., None, None]).to(torch.float8_e4m3fn)
    w, t = new | (old & new.any(-1, keepdim=True)), new.any(-1)
    pages.view(torch.uint8)[row[w]] = v.view(torch.uint8)[w]
    scales[blk[t]] = sc[t]
    i, b2 = s["idx"].long(), b[:, :, 0]
    at = s["table"].long()[b2, i.clamp(min=0) // page] * page + i.clamp(min=0) % page
    got = pages[at].float() * scales[at // block][..., None]
    return [torch.where((i >= 0)[..., None], got, s["out"].float()).to(torch.bfloat16), s["scales"]]


def _lowest_free(refs, want):
    """The page of each wanted place (a truth value each), the lowest free pages in order; -1 elsewhere."""
    free = torch.nonzero(refs == 0).view(-1)
    k = torch.cumsum(want.view(-1).long(), 0) - 1
    return torch.where(want.view(-1), free[k.clamp(0, max(0, free.numel() - 1))], torch.full_like(k, -1)).view(want.shape)


def _fork(s):
    if own:
        s["ops"].pages_fork(s["book"], s["caches"], s["parent"], s["entries"])
        s["ops"].pages_reserve(s["book"], s["after"])
        return [s["table"], s["refs"], s["scales"], s["pages"].view(torch.uint8)] + ([s["index"]] if "index" in s else [])
    page, R, MP = s["case"]["page"], *s["table"].shape
    dev = s["table"].device
    par, r, lp = s["parent"].long(), torch.arange(R, device=dev), torch.arange(MP, device=dev)
    need = -(-s["entries"].long()[par] // page)
    new = torch.where((par == r)[:, None] | (lp[None, :] < need[:, None]), s["table"][par], torch.full_like(s["table"], -1)).long()
    # the last page is shared no further where it is partly filled: the parent's own slot keeps it, the others get copies
    copies = (par != r) & (s["entries"].long()[par] % page != 0)
    src = new[r, (need - 1).clamp(min=0)]
    new[r[copies], need[copies] - 1] = -1
    refs = s["refs"].long() - torch.bincount(s["table"][s["table"] >= 0].long(), minlength=s["refs"].numel())
    refs = refs + torch.bincount(new[new >= 0], minlength=refs.numel())
    dst = _lowest_free(refs, copies)
    new[r[copies], need[copies] - 1] = dst[copies]
    refs[dst[copies]] = 1
    for pool in [s["pages"].view(torch.uint8), s["scales"]] + ([s["index"]] if "index" in s else []):
        pool[dst[copies]] = pool[src[copies]]
    want = (new < 0) & (lp[None, :] < -(-s["after"].long()[:, None] // page))
    more = _lowest_free(refs, want)
    refs[more[want]] = 1
    s["table"].copy_(torch.where(want, more, new))
    s["refs"].copy_(refs)
    return [s["table"], s["refs"], s["scales"], s["pages"].view(torch.uint8)] + ([s["index"]] if "index" in s else [])


def _compact(s):
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    if own:
        s["ops"].pages_compact(s["book"], s["caches"], s["map"], s["live"])
        return [s["table"], s["refs"], s["map"], s["live"], s["scales"], s["pages"].view(torch.uint8)]
    live = s["refs"] > 0
    n = live.sum()
    i = torch.arange(live.numel(), device=live.device)
    hole, high = torch.nonzero(~live & (i < n)).view(-1), torch.nonzero(live & (i >= n)).view(-1)
    to = torch.where(live, i, torch.full_like(i, -1))
    to[high] = hole
    s["map"].copy_(to)
    s["live"].copy_(n.view(1))
    for pool in (s["pages"].view(torch.uint8), s["scales"], s["refs"]):
        pool[hole] = pool[high]
    s["refs"][high] = 0
    s["table"].copy_(torch.where(s["table"] >= 0, to[s["table"].long().clamp(min=0)], s["table"].long()))
    return [s["table"], s["refs"], s["map"], s["live"], s["scales"], s["pages"].view(torch.uint8)]


def _indexer(s):
    c = s["case"]
    if own:
        return s["ops"].indexer_scores_paged(s["q_pos"], s["q"], s["w"], s["caches"][0], ratio=c["ratio"], scores=s["scores"], ws=s["ws"])
    B, MP = s["table"].shape
    k = s["index"][s["table"].long().clamp(min=0)].float().view(B, 1, MP * c["page"], 128)
    x = torch.matmul(s["q"].float(), k.transpose(2, 3)).relu_().mul_(s["w"][..., None]).sum(2)
    seen = torch.arange(MP * c["page"], device=x.device) < ((s["q_pos"].long() + 1) // c["ratio"])[..., None]
    s["scores"].copy_(torch.where(seen, x, s["scores"]))
    return s["scores"]


# ------------------------------------------------------------------------------------------------ work and exact values


def work(case):
    k, page = case["kind"], case["page"]
    if k == "attention":
        nq, W, H = case["B"] * case["S"], case["window"], case["H"]
        vis = max(0, case["ctx"] - case["S"] // 2) // case["ratio"]
        n = min(case["topk"], vis) if case["topk"] else vis
        w = min(W, case["ctx"])
        # a segment's queries share their rows: what it cannot do without is each row once
        ent = case["B"] * (n if case["S"] == 1 else min(vis, n * case["S"]))
        win = case["B"] * (w if case["S"] == 1 else min(case["ctx"], case["S"] + W))
        byt = ent * (D + 4.0 / case["block"]) + win * D * 2 + nq * (H * D * 4 + case["topk"] * 4)
        return dict(bytes=byt, flops=4.0 * H * nq * (w + n) * D)
    if k == "append":
        n = case["B"] * max(1, case["S"] // case["ratio"])
        old = case["B"] * (case["block"] - 1) / 2
        return dict(bytes=n * (D * 2 + D) + (n + old) * (D + D * 2) + (n + old) / case["block"] * 8, flops=6.0 * n * D)
    if k == "fork":
        copied = (case["slots"] - case["groups"]) * (page * D / 2 + page / case["block"] * 2 + (page * 128 if case["pools"] == 2 else 0))
        return dict(bytes=2 * copied + case["slots"] * 4.0 * (case["entries"] / page + 2) * 2, flops=0)
    if k == "compact":
        moved = case["pages"] * min(1.0, case["live"]) * (1 - min(1.0, case["live"]))
        return dict(bytes=2 * moved * (page * D + page / case["block"] * 4) + case["pages"] * 4.0 * 6, flops=0)
    nq, vis = case["B"] * case["S"], max(1, case["ctx"] // case["ratio"])
    return dict(bytes=case["B"] * vis * 256 + nq * (case["HI"] * 260 + vis * 4), flops=2.0 * nq * case["HI"] * vis * 128)


def exact(case, seed):
    if case["kind"] in ("fork", "compact"):
        return None
    s = prepare(case, seed)
    f64 = torch.float64
    if case["kind"] == "attention":
        return torch.stack([_exact_request(s, b) for b in range(case["B"])])
    if case["kind"] == "append":
        return _exact_append(s)
    B, MP = s["table"].shape
    k = s["index"][s["table"].long().clamp(min=0)].to(f64).reshape(B, MP * case["page"], 128)
    x = torch.einsum("bsh,bshe->bse", s["w"].to(f64), torch.einsum("bshd,bed->bshe", s["q"].to(f64), k).clamp(min=0))
    seen = torch.arange(x.shape[-1], device=x.device) < ((s["q_pos"].long() + 1) // case["ratio"])[..., None]
    return x * seen


def _exact_request(s, b):
    """Request b's attention: its entries laid out densely, the sink as one more column of a softmax, the rotation in complex numbers."""
    c, f64, t = s["case"], torch.float64, s["q_pos"][b].long()
    held = s["table"][b].long().clamp(min=0)
    dense = s["pages"][held].reshape(-1, D)
    scale = s["scales"][held].reshape(-1, 1).repeat_interleave(c["block"], 0)
    seen = torch.zeros(t.numel(), dense.shape[0] + 1, dtype=torch.bool, device=t.device)
    if s["topk"] is not None:
        seen.scatter_(1, s["topk"][b].long() % (dense.shape[0] + 1), True)  # -1 falls into the column behind the last entry
    else:
        seen |= torch.arange(dense.shape[0] + 1, device=t.device)[None, :] < ((t + 1) // c["ratio"])[:, None]
    used = seen[:, :-1].any(0).nonzero().view(-1)
    back = torch.arange(max(0, int(t[0]) - c["window"] + 1), int(t[-1]) + 1, device=t.device)
    rows = torch.cat([s["ring"][b][back % s["ring"].shape[1]].to(f64), dense[used].to(f64) * scale[used].to(f64)])
    near = (back[None, :] <= t[:, None]) & (back[None, :] > t[:, None] - c["window"])
    z = torch.einsum("nhd,cd->nhc", s["q"][b].to(f64), rows) / D**0.5
    z = z.masked_fill(~torch.cat([near, seen[:, used]], 1)[:, None, :], -math.inf)
    z = torch.cat([z, s["sink"].to(f64)[None, :, None].expand(z.shape[0], -1, -1)], -1)
    o = torch.einsum("nhc,cd->nhd", torch.softmax(z, -1)[..., :-1], rows)
    turn = torch.polar(torch.ones(1, dtype=f64, device=o.device), -t.to(f64).view(-1, 1, 1) * BASE ** (-torch.arange(0, ROPE, 2, device=o.device, dtype=f64) / ROPE))
    o[..., D - ROPE :] = torch.view_as_real(torch.view_as_complex(o[..., D - ROPE :].reshape(*o.shape[:2], -1, 2)) * turn).flatten(-2)
    return o


def _pow2(k):
    """2^k in 64 bits, by its bits."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """x (64 bits, at most 448 in magnitude) to the nearest e4m3 value, ties to even."""
    step = _pow2(torch.frexp(x.abs().clamp(min=2.0**-6))[1] - 4)  # exact: ties are common
    return torch.round(x / step) * step


def _exact_append(s):
    """Request by request on a dense copy of its entries: the blocks from the one that holds the first new entry on."""
    c, out, scales = s["case"], s["out"].double(), s["scales"].double()
    block, page, ratio = c["block"], c["page"], c["ratio"]
    for b in range(c["B"]):
        t0 = int(s["start"][b])
        e0, e1 = t0 // ratio, (t0 + c["S"]) // ratio
        lo = e0 // block * block
        hi = -(-e1 // block) * block
        if e1 <= e0:
            hi = max(hi, lo + block)
        e = torch.arange(lo, hi, device="cuda")
        at = s["table"][b].long()[(e // page).clamp(max=s["table"].shape[1] - 1)] * page + e % page
        old = (s["pages"].view(-1, D)[at].double() * s["scales"].view(-1)[at // block].double()[:, None]).view(-1, block, D)
        x = s["rows"][b][e.clamp(max=s["rows"].shape[1] - 1)].double().view(-1, block, D)
        new = ((e >= e0) & (e < e1)).view(-1, block)
        amax = (x.abs() * new[..., None]).flatten(1).amax(1)
        k = torch.ceil(torch.log2(amax / E4M3_MAX) - 1e-9).clamp(min=-100)  # bf16 maxima: the next above 448 * 2^k is 2^-8 away
        before = s["scales"].view(-1)[at.view(-1, block)[:, 0] // block].double()
        has = (e < e0).view(-1, block).any(1)
        sc = torch.where(new.any(1), torch.maximum(_pow2(k), torch.where(has, before, 0.0 * before)), before)
        v = _e4m3(torch.where(new[..., None], x, old) / sc[:, None, None]) * sc[:, None, None]
        scales.view(-1)[at.view(-1, block)[:, 0][new.any(1)] // block] = sc[new.any(1)]
        i = s["idx"][b].long()
        out[b][i >= 0] = v.reshape(-1, D)[i[i >= 0] - lo]
    return [out, scales]
