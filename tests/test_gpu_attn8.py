"""Attention over an 8-bit cache in pages (sparse_attn8, hca_attn8) against the float64 oracle on the dequantised cache."""

import math

import numpy as np
import pytest
import torch

from oracle import csa_oracle as O
from tests.parity import np64

pytestmark = pytest.mark.gpu

BOUNDS = 6
D = 512


@pytest.fixture(scope="module")
def ops():
    from long_context_decode_c4a_b200 import ops
    return ops


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_cache(ops, g, B, max_entries, page, block, spread=0.0):
    """A cache with random codes; scales powers of two around 2^-6, e^(spread * normal) apart."""
    max_pages = -(-max_entries // page)
    num_pages = B * max_pages + 3
    perm = torch.randperm(num_pages, generator=g)[: B * max_pages].to(torch.int32).view(B, max_pages).cuda()
    book = ops.PageTable(perm, torch.ones(num_pages, dtype=torch.int32, device="cuda"), page)
    scales = 2.0 ** torch.round(-7 + spread * torch.randn(num_pages, page // block, generator=g))
    codes = (torch.randn(num_pages, page, D, generator=g) * 100).clamp(-448, 448)
    return ops.PagedCache(book, codes.to(torch.float8_e4m3fn).cuda(), scales.cuda())


def dense(cache):
    """[B, max_entries, 512] values and their scales, in float64."""
    t = cache.book.table.long().cpu()
    ok = (t >= 0) & (t < cache.book.num_pages)
    codes = cache.pages.float().double().cpu()[t.clamp(0, cache.book.num_pages - 1)].flatten(1, 2).numpy()
    s = cache.scales.double().cpu().repeat_interleave(cache.block, 1)[t.clamp(0, cache.book.num_pages - 1)].flatten(1, 2).numpy()
    mapped = ok.repeat_interleave(cache.book.page_size, 1).numpy()
    return codes * s[..., None], s, mapped


def make_q(g, *shape):
    x = torch.randn(*shape, generator=g)
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


def reference(q, t, W, ring, cache, scales, selected, sink, scale, rope_dim, rope_base):
    """The oracle's output of one query, how far the kernel may be from it, from the roundings that it makes, and the mean of
    sum (w c)^2 over the output:
      a weight P is off by 2^-8 of itself, or where that is less by 2^-22 with the largest P (P holds the scale of its column) at
      2^-5 or more, and by 2^-4 of itself or 2^-25 at most;
      a score by 2^-21 max|q| sum|c| (q's second piece), 2^-17 max|c| sum|q| (a window row's), 1024 additions
      of fp32 (2^-23 each) and the rounding of the exponent's argument;
      O by its additions in fp32 (2^-23 each), a window value by 2^-17 of its row's largest.
    """
    cap = ring.shape[0]
    selected = [s for s in selected if s >= 0]
    win = [ring[p % cap] for p in O.window_positions(t, W)] if t >= 0 else []
    c = np.array(win + [cache[s] for s in selected]).reshape(-1, D)
    s = np.array([2.0 ** math.ceil(math.log2(max(np.max(np.abs(r)), 1e-30) / 448)) for r in win] + [scales[e] for e in selected])
    if len(c) == 0:
        return np.zeros_like(q), np.zeros_like(q), 0.0
    with np.errstate(all="ignore"):
        out = O.mqa_with_sink(q, c, sink, scale)
        l = scale * q @ c.T
        m = np.maximum(l.max(1), sink)
        w = np.exp(l - m[:, None])
        w /= (w.sum(1) + np.exp(sink - m))[:, None]
        n, nw = len(c), len(win)
        ac, aq = np.abs(c), np.abs(q)
        dl = abs(scale) * (2.0 ** -13 * aq @ ac.T + 2.0 ** -21 * aq.max(1)[:, None] * ac.sum(1))
        dl[:, :nw] += abs(scale) * 2.0 ** -17 * ac[:nw].max(1, initial=0) * aq.sum(1)[:, None]
        dl += 2.0 ** -22 * (np.abs(l) + np.abs(m)[:, None] + 32) + 2.0 ** -21
        rel = n * 2.0 ** -23 + dl + (w * dl).sum(1, keepdims=True)
        p, codes = w * s, ac / np.where(s == 0, 1, s)[:, None]
        unit = p.max(1, keepdims=True) * 2.0 ** 5
        tol = (w * rel) @ ac + np.maximum(2.0 ** -8 * p, np.minimum(2.0 ** -22 * unit, 2.0 ** -4 * p + 2.0 ** -25 * unit)) @ codes
        tol += (w[:, :nw] * 2.0 ** -17) @ np.repeat(ac[:nw].max(1, initial=0)[:, None], D, 1)
    r0 = D - rope_dim
    pair = tol[:, r0:].reshape(len(q), -1, 2).sum(-1, keepdims=True).repeat(2, -1).reshape(len(q), -1)
    tol[:, r0:] = pair + 2.0 ** -20 * np.abs(out[:, r0:]).max(1, initial=0)[:, None]
    return O.rope(out, t, rope_dim, rope_base, inverse=True), tol, np.mean(w ** 2 @ c ** 2)


def check_close(out, ref, tol, what):
    got = np64(out)
    tol = tol + 2.0 ** -24 * np.abs(ref)
    if out.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -9 * np.abs(ref) * (1 + 2.0 ** -8)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} beyond the bound, worst {np.nanmax(np.abs(got - ref) / tol):.2f} of it"


def run_case(ops, *, B, S, H, W, page, block, pos, topk=0, ratio=4, cap=None, spread=0.0, dtype=torch.bfloat16, seed=0, rope_dim=64,
             max_entries=None):
    """Positions pos[b] .. pos[b] + S - 1; `topk` random visible entries a query (0: every one)."""
    g = torch.Generator().manual_seed(seed)
    ents = max_entries or max(1, max((p + S) // ratio for p in pos))
    cache = make_cache(ops, g, B, ents, page, block, spread)
    q_pos = torch.tensor(pos, dtype=torch.int32)[:, None] + torch.arange(S, dtype=torch.int32)
    q = make_q(g, B, S, H, D)
    cap = cap or (W if S == 1 else W + S - 1)
    ring = torch.randn(B, cap, D, generator=g).to(torch.bfloat16)
    sink = torch.randn(H, generator=g)
    out = torch.full((B, S, H, D), 77.0, dtype=dtype, device="cuda")
    idx = None
    if topk:
        idx = torch.full((B, S, topk), -1, dtype=torch.int32)
        for b in range(B):
            for i in range(S):
                vis = max(0, (int(q_pos[b, i]) + 1) // ratio)
                sel = torch.randperm(vis, generator=g)[:topk]
                at = torch.randperm(topk, generator=g)[: sel.numel()]   # anywhere in the list, in any order
                idx[b, i, at] = sel.to(torch.int32)
        ws = ops.workspace(ops._lib.CSA_WS_SPARSE_ATTN, B, S, 1, 1)
        ops.sparse_attn8(q_pos.cuda(), q.cuda(), ring.cuda(), cache, idx.cuda(), sink.cuda(), W, ratio=ratio, out=out, rope_dim=rope_dim, ws=ws)
    else:
        ws = ops.workspace(ops._lib.CSA_WS_HCA_ATTN, B, S, 1, 1)
        ops.hca_attn8(q_pos.cuda(), q.cuda(), ring.cuda(), cache, sink.cuda(), W, ratio=ratio, out=out, rope_dim=rope_dim, ws=ws)
    assert ops.device_status(ws) == 0
    vals, scales, _ = dense(cache)
    for b in range(B):
        for i in range(S):
            t = int(q_pos[b, i])
            sel = idx[b, i].tolist() if topk else list(range((t + 1) // ratio))
            ref, tol, var = reference(np64(q[b, i]), t, W, np64(ring[b]), vals[b], scales[b], sel, np64(sink), 1 / math.sqrt(D), rope_dim, 10000.0)
            check_close(out[b, i], ref, tol, f"b={b} t={t}")
            if dtype == torch.float32 and spread == 0:
                # Independent roundings of the weights, each within 2^-8, have a variance of at most 2^-16 sum w^2 c^2
                # (uniform ones a third of it); the bounds above add them up in magnitude and are never near.
                assert np.mean((np64(out[b, i]) - ref) ** 2) <= 2.0 ** -16 * var


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,S,H,W,page,block,pos,topk", [
    (1, 1, 128, 128, 64, 16, [0], 4),                # the first token: one window row, no entry
    (1, 1, 128, 128, 64, 16, [3], 4),                # the first entry
    (2, 1, 128, 128, 64, 16, [4095, 700], 1024),
    (1, 1, 8, 16, 16, 1, [77], 7),
    (3, 1, 100, 100, 32, 4, [300, 131, 64], 65),     # tiles and pages that end inside one another
    (1, 1, 1, 1, 128, 64, [2000], 64),
    (80, 1, 128, 33, 16, 16, [900 + 3 * i for i in range(80)], 200),   # one pair of CTAs a query
    (1, 90, 64, 128, 64, 8, [0], 20),                # a segment from the start of a prompt
    (2, 40, 128, 200, 64, 2, [55, 700], 2048),
])
def test_list(ops, B, S, H, W, page, block, pos, topk, dtype):
    run_case(ops, B=B, S=S, H=H, W=W, page=page, block=block, pos=pos, topk=topk, dtype=dtype)


@pytest.mark.parametrize("B,S,H,W,page,block,pos,ratio", [
    (1, 1, 128, 128, 64, 16, [5], 128),              # no entry yet
    (1, 1, 128, 128, 32, 1, [200002], 128),
    (3, 1, 64, 128, 64, 32, [127, 128, 9000], 128),
    (1, 1, 128, 16, 16, 2, [19999], 4),              # 5000 entries: more than a list holds
    (75, 1, 128, 128, 1024, 64, [5000 + i for i in range(75)], 4),
    (1, 50, 32, 128, 64, 16, [350], 4),
    (1, 39, 128, 100, 64, 16, [380], 4),
])
def test_range(ops, B, S, H, W, page, block, pos, ratio):
    run_case(ops, B=B, S=S, H=H, W=W, page=page, block=block, pos=pos, ratio=ratio)


@pytest.mark.parametrize("spread", [1.0, 4.0])
def test_scales_far_apart(ops, spread):
    run_case(ops, B=2, S=1, H=128, W=64, page=32, block=2, pos=[2000, 1234], topk=300, spread=spread, dtype=torch.float32)


def test_wide_window_and_rope(ops):
    run_case(ops, B=1, S=3, H=16, W=1024, page=64, block=16, pos=[3000], topk=64, dtype=torch.float32, rope_dim=128)
    run_case(ops, B=1, S=1, H=16, W=700, page=64, block=16, pos=[650], topk=64, cap=999, rope_dim=2)


# ------------------------------------------------------------------------------------------------ hard rows


class Plain:
    """One request, every entry of a 64-entry page table visible; the test changes what it wants."""

    def __init__(self, ops, E=640, W=16, H=128, t=None, seed=1):
        g = torch.Generator().manual_seed(seed)
        self.ops, self.W, self.t = ops, W, 4 * E - 1 if t is None else t
        self.cache = make_cache(ops, g, 1, E, 64, 16)
        self.q, self.ring, self.sink = make_q(g, 1, 1, H, D), torch.randn(1, W, D, generator=g).to(torch.bfloat16), torch.randn(H, generator=g)
        self.idx = torch.arange(E, dtype=torch.int32).view(1, 1, E)
        self.ws = ops.workspace(ops._lib.CSA_WS_SPARSE_ATTN, 1, 1, 1, 1)

    def run(self, split=True, form="list", scale=None):
        out = torch.full(self.q.shape, 77.0, dtype=torch.float32, device="cuda")
        ws = self.ws if split else self.ws[:256]
        args = (i32([[self.t]]), self.q.cuda(), self.ring.cuda(), self.cache)
        if form == "list":
            self.ops.sparse_attn8(*args, self.idx.cuda(), self.sink.cuda(), self.W, out=out, ws=ws, scale=scale)
        else:
            self.ops.hca_attn8(*args, self.sink.cuda(), self.W, ratio=4, out=out, ws=ws, scale=scale)
        return out[0, 0]

    def want(self, selected=None, scale=1 / math.sqrt(D)):
        vals, s, _ = dense(self.cache)
        sel = self.idx.view(-1).tolist() if selected is None else selected
        return reference(np64(self.q[0, 0]), self.t, self.W, np64(self.ring[0]), vals[0], s[0], sel, np64(self.sink), scale, 64, 10000.0)

    def check(self, selected=None, status=0, forms=("list", "range"), scale=None):
        for split in (True, False):
            for form in forms:
                out = self.run(split, form, scale)
                assert self.ops.device_status(self.ws) == status
                ref, tol, _ = self.want(selected, scale or 1 / math.sqrt(D))
                check_close(out, ref, tol, f"{form} split={split}")


@pytest.mark.parametrize("W", [1, 33, 97, 128])
@pytest.mark.parametrize("E", [1, 64, 65, 129, 200, 257, 321, 400, 449, 520, 577, 700, 800])
def test_every_number_of_tiles(ops, E, W):
    """1 to 17 tiles, whole and split, odd and even numbers of them on each CTA of a pair, any mix of window and entries."""
    Plain(ops, E=E, W=W, H=32, t=4 * E + 130, seed=E + W).check(forms=("list",))   # (more are visible than the list has)
    Plain(ops, E=E, W=W, H=32, t=4 * E + 2, seed=E + W + 1).check(forms=("range",))


def test_rising_logits(ops):
    """Scores that climb by far more than the kernel's headroom, tile after tile and row by row."""
    p = Plain(ops)
    vals = (p.q[0, 0, 0].float() * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    t = p.cache.book.table[0].long()
    for i in range(10):
        p.cache.pages.view(torch.uint8)[t[i]] = vals.view(torch.uint8).cuda()
        p.cache.scales[t[i]] = 2.0 ** (i - 9)
    p.check()
    p.q[0, 0, 1::2] = -p.q[0, 0, 1::2]     # and fall, for half of the heads
    p.check()


def test_one_large_weight_before_a_flat_tail(ops):
    """One entry of weight near 1, thousands of 2^-17 each: together they count."""
    p = Plain(ops, E=8192)
    t = p.cache.book.table[0].long()
    u = torch.ones(512)
    u[1::2] = -1
    p.q[0, 0] = u.to(torch.bfloat16)
    p.ring.zero_()
    p.sink.fill_(float("-inf"))
    g = torch.Generator(device="cuda").manual_seed(0)
    noise = torch.randint(0, 2, (p.cache.pages.shape[0], 64, 256), device="cuda", generator=g) * 2.0 - 1
    p.cache.pages.copy_(noise.repeat_interleave(2, -1).to(torch.float8_e4m3fn))   # no part along q, values of +-1
    p.cache.scales.fill_(1.0)
    p.cache.pages[t[3], 7] = (u * 0.5).to(torch.float8_e4m3fn)                    # l = 0.5 sqrt(512) = 11.3: 2^16.3 to 1
    p.check(forms=("range",))


@pytest.mark.parametrize("scale", [-0.5, 0.0, 1e-6, 3.0])
def test_other_scales(ops, scale):
    p = Plain(ops, E=100)
    for split in (True, False):
        out = p.run(split, scale=scale)
        ref, tol, _ = p.want(scale=scale)
        check_close(out, ref, tol, f"scale={scale}")


def test_sinks(ops):
    p = Plain(ops, E=100)
    p.sink[:4] = torch.tensor([float("-inf"), 1e4, -1e4, 60.0])
    p.check()
    p.sink[5] = float("inf")
    for split in (True, False):
        out = p.run(split)
        assert (out[5] == 0).all() and out.isfinite().all()


def test_lists_that_leave_little(ops):
    p = Plain(ops, E=100)
    p.idx.fill_(-1)
    p.check(forms=("list",))                     # the window alone
    p.idx[0, 0, 57] = 99
    p.check(forms=("list",))
    p.idx[0, 0, 3:9] = 42                        # the same entry six times counts six times
    p.check(forms=("list",))


def test_padding_queries(ops):
    """A negative position: output zero, whatever its list holds; its neighbours are not disturbed."""
    g = torch.Generator().manual_seed(2)
    cache = make_cache(ops, g, 3, 200, 64, 16)
    q, ring, sink = make_q(g, 3, 1, 128, D).cuda(), torch.randn(3, 128, D, generator=g).to(torch.bfloat16).cuda(), torch.randn(128, generator=g).cuda()
    idx = torch.arange(200, dtype=torch.int32, device="cuda").expand(3, 1, 200).contiguous()
    idx[1].fill_(123456)
    a = ops.sparse_attn8(i32([[799], [-1], [799]]), q, ring, cache, idx, sink, 128)
    b = ops.sparse_attn8(i32([[799], [799], [799]]), q, ring, cache, idx, sink, 128)
    assert (a[1] == 0).all() and torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    h = ops.hca_attn8(i32([[799], [-5], [799]]), q, ring, cache, sink, 128, ratio=4)
    assert (h[1] == 0).all() and (h[0] != 0).any()


def test_bad_pages_and_entries(ops):
    """Entries that are not visible, behind the table or on missing pages are left out and reported."""
    p = Plain(ops, E=640)
    t0 = p.cache.book.table.clone()
    p.cache.book.table[0, 2] = -1
    p.cache.book.table[0, 5] = p.cache.book.num_pages
    keep = [e for e in range(640) if e // 64 not in (2, 5)]
    p.check(keep, status=BOUNDS)
    p.cache.book.table.copy_(t0)
    p.t = 4 * 500 - 1                            # entries 500 .. 639 are not visible
    p.check(list(range(500)), status=BOUNDS, forms=("list",))
    p.idx = p.idx[..., :500].contiguous()
    p.check(list(range(500)))
    p.idx[0, 0, 7] = 2 ** 31 - 1
    p.check([e for e in range(500) if e != 7], status=BOUNDS, forms=("list",))
    p.t = 4 * 700                                # 700 entries visible, the table has places for 640
    p.check(list(range(640)), status=BOUNDS, forms=("range",))


def test_what_is_not_a_number(ops):
    """NaN and infinities reach the heads and queries that read them, and no others; masked rows may hold anything."""
    p = Plain(ops, E=256)
    t = p.cache.book.table[0].long()
    ref = p.run()
    p.cache.pages.view(torch.uint8)[t[1]] = 0x7F           # NaN codes on a page that the list leaves out
    p.cache.scales[t[2]] = float("nan")
    p.idx = torch.cat([torch.arange(64), torch.arange(192, 256)]).to(torch.int32).view(1, 1, -1)
    p.check(forms=("list",))
    p.idx = torch.cat([p.idx, torch.tensor([[[130]]], dtype=torch.int32)], -1)
    for split in (True, False):
        assert p.run(split).isnan().all()
    p = Plain(ops, E=256)
    p.q[0, 0, 9, 100] = float("nan")
    p.q[0, 0, 10, 100] = float("inf")
    for split in (True, False):
        out = p.run(split)
        assert out[9].isnan().all() and out[10].isnan().all()
        rest = [h for h in range(128) if h not in (9, 10)]
        assert out[rest].isfinite().all()
        assert torch.allclose(out[rest], ref[rest], rtol=0.05, atol=0.05)
    p = Plain(ops, E=256, W=16)
    p.ring[0, 5, 5] = float("nan")
    for split in (True, False):
        assert p.run(split).isnan().all()
    p = Plain(ops, E=256, W=16, t=3)                       # rows of the ring that no token has filled
    p.ring[0, 4:] = float("nan")
    p.idx = torch.zeros(1, 1, 1, dtype=torch.int32)
    p.check([0], forms=("list", "range"))


def test_zero_scales_do_not_count(ops):
    p = Plain(ops, E=128)
    t = p.cache.book.table[0].long()
    p.cache.scales[t[0], 1] = 0.0
    keep = [e for e in range(128) if not 16 <= e < 32]
    p.check(keep)


def test_extreme_magnitudes(ops):
    """q and rows near the ends of their ranges; tiny scales beside ordinary ones."""
    p = Plain(ops, E=128)
    t = p.cache.book.table[0].long()
    p.cache.scales[t[1]] = 2.0 ** -100
    p.check()
    p.q[0, 0, 3] *= 2.0 ** -90
    p.q[0, 0, 4] = 0
    p.ring[0, 2] = 0
    p.ring[0, 3] *= 2.0 ** -110
    p.check()


# ------------------------------------------------------------------------------------------------ the way of calling


def test_strides_streams_and_graphs(ops):
    """A ring that is a slice of a larger one; another stream; a captured step replayed on new contents."""
    g = torch.Generator().manual_seed(3)
    B, W, E = 3, 100, 300
    cache = make_cache(ops, g, B, E, 64, 16)
    big = torch.randn(B, 150, D, generator=g).to(torch.bfloat16).cuda()
    ring = big[:, :120]
    q, sink = make_q(g, B, 1, 128, D).cuda(), torch.randn(128, generator=g).cuda()
    idx = torch.stack([torch.randperm(E, generator=g)[:77] for _ in range(B)]).to(torch.int32).view(B, 1, 77).cuda()
    pos = i32([[4 * E + 1]] * B)
    ws = ops.workspace(ops._lib.CSA_WS_SPARSE_ATTN, B, 1, 1, 1)
    want = ops.sparse_attn8(pos, q, ring.contiguous(), cache, idx, sink, W, ws=ws)
    assert torch.equal(ops.sparse_attn8(pos, q, ring, cache, idx, sink, W, ws=ws), want)
    off = torch.empty(q.numel() + 8, dtype=torch.bfloat16, device="cuda")[8:].view(q.shape)   # 16 bytes past a multiple of 32
    assert torch.equal(ops.sparse_attn8(pos, q, ring, cache, idx, sink, W, ws=ws[:256], out=off),
                       ops.sparse_attn8(pos, q, ring, cache, idx, sink, W, ws=ws[:256]))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert torch.equal(ops.sparse_attn8(pos, q, ring, cache, idx, sink, W, ws=ws), want)
    torch.cuda.synchronize()
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.sparse_attn8(pos, q, ring, cache, idx, sink, W, out=out, ws=ws)
        again = ops.hca_attn8(pos, q, ring, cache, sink, W, ratio=4, ws=ws)
    graph.replay()
    assert torch.equal(out, want)
    q.copy_(make_q(g, B, 1, 128, D))
    pos.fill_(903)
    graph.replay()
    assert torch.equal(again, ops.hca_attn8(pos, q, ring, cache, sink, W, ratio=4, ws=ws))


def test_rows_past_32_bits(ops):
    """Pages more than 4 GB into the pool."""
    num_pages = 140000
    book = ops.PageTable.empty(1, 8, num_pages, 64)
    book.table.copy_(i32([[num_pages - 1 - 9999 * i for i in range(8)]]))
    cache = ops.PagedCache.e4m3(book, block=16)
    g = torch.Generator().manual_seed(4)
    for p in book.table[0].tolist():
        cache.pages[p] = (torch.randn(64, D, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
        cache.scales[p] = 2.0 ** -6
    q, ring, sink = make_q(g, 1, 1, 128, D), torch.randn(1, 16, D, generator=g).to(torch.bfloat16), torch.randn(128, generator=g)
    out = ops.hca_attn8(i32([[2047]]), q.cuda(), ring.cuda(), cache, sink.cuda(), 16, ratio=4)
    vals = (cache.pages[book.table[0].long()].float() * 2.0 ** -6).double().cpu().flatten(0, 1).numpy()
    ref, tol, _ = reference(np64(q[0, 0]), 2047, 16, np64(ring[0]), vals, np.full(512, 2.0 ** -6), range(512), np64(sink), 1 / math.sqrt(D), 64, 10000.0)
    check_close(out[0, 0], ref, tol, "far pages")
