"""The caches in pages on the GPU: page-table calls, appends, reads and index scores, against the oracle."""

import numpy as np
import pytest
import torch

from oracle import csa_oracle as O
from oracle import paged_oracle as PO
from tests.parity import check_topk, np64

pytestmark = pytest.mark.gpu

BOUNDS, NO_PAGES = 6, 7


@pytest.fixture(scope="module")
def ops():
    from long_context_decode_c4a_b200 import ops
    return ops


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def random_book(ops, g, slots, max_pages, num_pages, page, used):
    """Slot r maps its first used[r] places to random pages."""
    perm = torch.randperm(num_pages, generator=g).tolist()
    table = [[perm.pop() if lp < used[r] else -1 for lp in range(max_pages)] for r in range(slots)]
    refs = [0] * num_pages
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    return ops.PageTable(i32(table), i32(refs), page), table, refs


def same_book(book, table, refs):
    assert book.table.tolist() == table
    assert book.refs.tolist() == refs


# ------------------------------------------------------------------------------------------------ page table


@pytest.mark.parametrize("slots,max_pages,page", [(1, 1, 16), (3, 5, 16), (64, 130, 64), (700, 13, 1024), (1, 20000, 64), (2100, 5, 16)])
def test_reserve(ops, slots, max_pages, page):
    g = torch.Generator().manual_seed(slots)
    used = torch.randint(0, max_pages + 1, (slots,), generator=g).tolist()
    num_pages = slots * max_pages
    book, table, refs = random_book(ops, g, slots, max_pages, num_pages, page, used)
    entries = torch.randint(0, max_pages * page + 1, (slots,), generator=g).tolist()
    ops.pages_reserve(book, i32(entries))
    PO.reserve(table, refs, page, entries)
    same_book(book, table, refs)
    assert ops.device_status(book.ws) == 0


def test_reserve_without_enough_pages_changes_nothing(ops):
    book = ops.PageTable.empty(2, 4, 5, 16)
    ops.pages_reserve(book, i32([64, 32]))
    assert ops.device_status(book.ws) == NO_PAGES
    same_book(book, [[-1] * 4] * 2, [0] * 5)
    ops.pages_reserve(book, i32([64, 16]))   # just enough
    assert ops.device_status(book.ws) == 0
    same_book(book, [[0, 1, 2, 3], [4, -1, -1, -1]], [1] * 5)


@pytest.mark.parametrize("entries", [[-1, 0], [0, 65]])
def test_reserve_out_of_range(ops, entries):
    book = ops.PageTable.empty(2, 4, 8, 16)
    ops.pages_reserve(book, i32(entries))
    assert ops.device_status(book.ws) == BOUNDS
    same_book(book, [[-1] * 4] * 2, [0] * 8)


@pytest.mark.parametrize("seed,slots,max_pages,page", [(0, 1, 3, 16), (1, 4, 3, 16), (2, 9, 7, 32), (3, 64, 40, 64), (4, 300, 9, 16), (5, 2500, 3, 16)])
def test_fork_keep_free(ops, seed, slots, max_pages, page):
    """Random parent maps (kept, copied, swapped and freed slots), several in a row, with the rows that follow the pages."""
    g = torch.Generator().manual_seed(seed)
    entries = torch.randint(0, max_pages * page + 1, (slots,), generator=g).tolist()
    used = [min(max_pages, -(-e // page) + int(torch.randint(0, 2, (1,), generator=g))) for e in entries]
    num_pages = 2 * slots * max_pages
    book, table, refs = random_book(ops, g, slots, max_pages, num_pages, page, used)
    refs[5 % num_pages] += 1  # held from outside
    book.refs[5 % num_pages] += 1
    caches = [ops.PagedCache.e4m3(book, block=16), ops.PagedCache.bf16(book, 128), ops.PagedCache.e4m3(book, block=1), ops.PagedCache.bf16(book, 24)]
    gg = torch.Generator(device="cuda").manual_seed(seed)
    for c in caches:
        raw = torch.randint(0, 256, (c.pages.numel() * c.pages.element_size(),), dtype=torch.uint8, device="cuda", generator=gg)
        c.pages.view(torch.uint8).view(-1).copy_(raw)
        if c.scales is not None:
            c.scales.uniform_(generator=gg)
    for _ in range(3):
        parent = torch.randint(-1, slots, (slots,), generator=g).tolist()
        parent = [r if torch.rand((), generator=g) < 0.3 else p for r, p in enumerate(parent)]
        want = [[t.clone() for t in (c.pages.view(torch.uint8), c.scales) if t is not None] for c in caches]
        ops.pages_fork(book, caches, i32(parent), i32(entries))
        moves = PO.fork(table, refs, page, parent, entries)
        same_book(book, table, refs)
        for c, pools in zip(caches, want):
            for pool, now in zip(pools, (c.pages.view(torch.uint8), c.scales)):
                for a, b in moves:
                    pool[b] = pool[a]
                assert torch.equal(pool, now)
        entries = [entries[p] if p >= 0 else 0 for p in parent]
    assert ops.device_status(book.ws) == 0


@pytest.mark.parametrize("slots", [4, 2500])  # the slots' arguments in shared memory, in the workspace
@pytest.mark.parametrize("places", [1, 1100])  # one CTA, a cluster
@pytest.mark.parametrize("table,outside,parent,entries", [
    ([0, 0, -1, -1], 0, [-1, 1, 0, -1], [9, 16, 0, 0]),     # another slot has all 16 rows
    ([0, -1, -1, -1], 1, [-1, 0, 0, -1], [9, 0, 0, 0]),     # a holder outside the table
    ([0, 0, -1, -1], 0, [-1, -1, 1, 0], [9, 7, 0, 0]),      # two parents of one page
    ([0, 0, -1, -1], 0, [-1, -1, 1, 0], [16, 7, 0, 0]),     # a copy that takes it whole, one that does not
])
def test_fork_keeps_no_page_that_another_has(ops, slots, places, table, outside, parent, entries):
    """Rows appended behind a copy's entries meet nobody else's."""
    rows = [[p] + [-1] * (places - 1) for p in table] + [[-1] * places for _ in range(slots - 4)]
    refs = [sum(p == 0 for p in table) + outside] + [0] * 7
    book = ops.PageTable(i32(rows), i32(refs), 16)
    cache = ops.PagedCache.bf16(book, 8)
    cache.pages[0] = torch.arange(16, device="cuda")[:, None].to(torch.bfloat16)
    pad = [-1] * (slots - 4)
    moves = PO.fork(rows, refs, 16, parent + pad, entries + [0] * (slots - 4))
    ops.pages_fork(book, [cache], i32(parent + pad), i32(entries + [0] * (slots - 4)))
    same_book(book, rows, refs)
    assert len(moves) == (2 if outside else 1)  # a holder outside: neither heir keeps the page
    for src, dst in moves:
        assert src == 0 and torch.equal(cache.pages[dst], cache.pages[0])
    # Slot r's new rows (its number) behind what it took over.
    start = [-1 if p < 0 or p == r else entries[p] for r, p in enumerate(parent)]
    start = [e if 0 <= e < 16 else -1 for e in start]
    new = torch.arange(4, device="cuda").view(4, 1, 1).expand(4, 16, 8).contiguous().to(torch.bfloat16) + 100
    ops.cache_append(cache, i32(start), 1, new, 1)
    assert ops.device_status(book.ws) == 0
    for r, p in enumerate(parent):
        if p >= 0:
            n = entries[p]
            want = list(range(n)) + ([100 + r] if start[r] >= 0 else [])
            got = ops.cache_read(cache, i32([list(range(len(want))) if s == r else [-1] * len(want) for s in range(4)]))[r, :, 0]
            assert got.tolist() == want


def test_fork_needs_pages(ops):
    book = ops.PageTable.empty(4, 2, 3, 16)
    ops.pages_reserve(book, i32([20, 0, 0, 0]))
    before = book.table.tolist(), book.refs.tolist()
    ops.pages_fork(book, [], i32([0, 0, 0, -1]), i32([20, 0, 0, 0]))   # two copies, one free page
    assert ops.device_status(book.ws) == NO_PAGES
    same_book(book, *before)
    ops.pages_fork(book, [], i32([0, 0, -1, -1]), i32([20, 0, 0, 0]))
    assert ops.device_status(book.ws) == 0
    same_book(book, [[0, 1], [0, 2], [-1, -1], [-1, -1]], [2, 1, 1])
    ops.pages_fork(book, [], i32([-1, 1, -1, -1]), i32([20, 20, 0, 0]))  # the first leaves: the shared page stays
    same_book(book, [[-1, -1], [0, 2], [-1, -1], [-1, -1]], [1, 0, 1])


@pytest.mark.parametrize("parent,entries", [([2, 0], [0, 0]), ([-2, 0], [0, 0]), ([0, 1], [33, 0]), ([0, 1], [-1, 0])])
def test_fork_out_of_range(ops, parent, entries):
    book = ops.PageTable.empty(2, 2, 8, 16)
    ops.pages_reserve(book, i32([17, 0]))
    before = book.table.tolist(), book.refs.tolist()
    ops.pages_fork(book, [], i32(parent), i32(entries))
    assert ops.device_status(book.ws) == BOUNDS
    same_book(book, *before)


@pytest.mark.parametrize("live", [0.0, 0.1, 0.5, 0.9, 1.0])
@pytest.mark.parametrize("num_pages", [1, 37, 9001])
def test_compact(ops, num_pages, live):
    g = torch.Generator().manual_seed(num_pages)
    slots = min(num_pages, 8)
    max_pages = num_pages // slots
    used = [int(round(live * max_pages))] * slots
    book, table, refs = random_book(ops, g, slots, max_pages, num_pages, 16, used)
    caches = [ops.PagedCache.e4m3(book, block=4), ops.PagedCache.bf16(book, 128)]
    gg = torch.Generator(device="cuda").manual_seed(1)
    caches[0].pages.view(torch.uint8).copy_(torch.randint(0, 256, caches[0].pages.shape, dtype=torch.uint8, device="cuda", generator=gg))
    caches[0].scales.uniform_(generator=gg)
    caches[1].pages.normal_(generator=gg)
    want = [caches[0].pages.view(torch.uint8).clone(), caches[0].scales.clone(), caches[1].pages.clone()]
    where, n = ops.pages_compact(book, caches)
    moves, ref_map, ref_live = PO.compact(table, refs)
    same_book(book, table, refs)
    assert where.tolist() == ref_map and n.item() == ref_live
    if moves:
        a, b = torch.tensor([m[0] for m in moves], device="cuda"), torch.tensor([m[1] for m in moves], device="cuda")
        for pool in want:
            pool[b] = pool[a]
    for pool, now in zip(want, [caches[0].pages.view(torch.uint8), caches[0].scales, caches[1].pages]):
        assert torch.equal(pool, now)
    assert ops.device_status(book.ws) == 0


def test_many_caches_follow(ops):
    """More caches than one copy launch takes (a model's layers behind one table)."""
    book = ops.PageTable.empty(2, 2, 6, 16)
    ops.pages_reserve(book, i32([20, 0]))
    caches = [ops.PagedCache.bf16(book, 8 * (1 + i % 3)) for i in range(131)]
    for i, c in enumerate(caches):
        c.pages.fill_(i + 1)
        c.pages[2:].zero_()
    ops.pages_fork(book, caches, i32([0, 0]), i32([20, 0]))
    same_book(book, [[0, 1], [0, 2]], [2, 1, 1, 0, 0, 0])
    for i, c in enumerate(caches):
        assert (c.pages[2] == i + 1).all() and (c.pages[3:] == 0).all()


# ------------------------------------------------------------------------------------------------ append, read


def values(cache):
    """The cache's values row by row, in float64 on the host."""
    x = cache.pages.float().double().cpu()
    if cache.scales is not None:
        x = x * cache.scales.double().cpu().repeat_interleave(cache.block, 1)[..., None]
    return x


@pytest.mark.parametrize("page,block", [(16, 1), (16, 16), (32, 4), (64, 32), (64, 64), (1024, 64), (128, 2)])
@pytest.mark.parametrize("ratio", [4, 128])
def test_append(ops, page, block, ratio):
    """Segments of many lengths one after another, the rows' magnitudes rising and falling, against the oracle."""
    g = torch.Generator().manual_seed(page * 131 + block + ratio)
    B, max_pages = 3, max(2, 256 // page)
    used = [max_pages] * B
    book, table, _ = random_book(ops, g, B, max_pages, B * max_pages + 2, page, used)
    c8, c16 = ops.PagedCache.e4m3(book, block=block), ops.PagedCache.bf16(book, 128)
    codes, scales = np.zeros((book.num_pages, page, 512)), np.zeros((book.num_pages, page // block))
    plain = np.zeros((book.num_pages, page, 128))
    pos = [0, 3, 7 * ratio + 2]
    cap = 150
    rows = torch.zeros(B, cap, 512, dtype=torch.bfloat16)
    for S in (1, ratio, 1, 2 * ratio + 1, 40 * ratio + 3, 1, ratio - 1, 17 * ratio):
        rows = (torch.randn(B, cap, 512, generator=g) * torch.exp(3 * torch.randn(B, cap, 1, generator=g))).to(torch.bfloat16)
        rows[:, ::7] = 0
        ops.cache_append(c8, i32(pos), S, rows.cuda(), ratio)
        ops.cache_append(c16, i32(pos), S, rows[..., :128].contiguous().cuda(), ratio)
        for b in range(B):
            e0, e1 = pos[b] // ratio, (pos[b] + S) // ratio
            PO.append(codes, scales, table[b], page, block, e0, e1, np64(rows[b]))
            for e in range(e0, e1):
                plain[table[b][e // page], e % page] = np64(rows[b, e, :128])
            pos[b] += S
        assert np.array_equal(np64(c8.scales), scales)
        assert np.array_equal(np64(c8.pages.float()), codes)
        assert np.array_equal(np64(c16.pages.float()), plain)
    assert ops.device_status(book.ws) == 0
    # read back, in any order, the same entry twice, gaps left alone
    n = 300
    idx = torch.stack([torch.randint(-1, p // ratio, (n,), generator=g) for p in pos]).to(torch.int32)
    for c, ref in ((c8, codes * np.repeat(scales, block, 1)[..., None]), (c16, plain)):
        out = torch.full((B, n, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
        ops.cache_read(c, idx.cuda(), out=out)
        got = np64(out)
        for b in range(B):
            for i, e in enumerate(idx[b].tolist()):
                want = ref[table[b][e // page], e % page] if e >= 0 else np.full(c.d, 7.0)
                assert np.array_equal(got[b, i], want)
    assert ops.device_status(book.ws) == 0


def test_append_extremes(ops):
    """Values at the ends of bf16's range, subnormals, zeros, infinities and NaN; padding requests; rows of a slice."""
    page = block = 16
    book = ops.PageTable.empty(4, 1, 4, page)
    ops.pages_reserve(book, i32([16, 16, 16, 16]))
    c = ops.PagedCache.e4m3(book, block=block)
    c.scales.fill_(5.0)   # stale: a block without earlier rows takes nothing from it
    rows = torch.zeros(4, 20, 512, dtype=torch.bfloat16)
    rows[0, 0] = torch.finfo(torch.bfloat16).max
    rows[0, 1, 3] = 1.0
    rows[1, 0, 0] = 1e-40     # subnormal
    rows[2, 0, 5] = float("inf")
    rows[3, 0] = 448.0
    rows[3, 1] = -449.0
    ops.cache_append(c, i32([0, 0, 0, -1]), 8, rows.cuda()[:, :9], 4)
    s = c.scales.view(-1).tolist()
    assert s[0] == 2.0 ** 120 and s[1] == 2.0 ** -100 and s[2] != s[2] and s[3] == 5.0
    got = values(c)
    # bf16's largest value 0x7F7F is 255 * 2^120: e4m3 of 255 is 256
    assert (got[0, 0] == 256 * 2.0 ** 120).all() and (got[0, 1] == 0).all()
    assert (got[1] == 0).all() and got[2, 0].isnan().all() and (c.pages[3].float() == 0).all()
    ops.cache_append(c, i32([-1, -1, 4, 0]), 8, rows.cuda(), 4)  # the NaN block stays NaN
    s = c.scales.view(-1).tolist()
    assert s[2] != s[2] and s[3] == 1.0   # 449 is a tie between 448 and 450 in bf16: 448
    assert values(c)[3, 0, 0] == 448 and values(c)[3, 1, 0] == -448
    rows[3, 2] = 450.0                           # beyond 448: the step doubles, the earlier rows stay on it
    ops.cache_append(c, i32([-1, -1, -1, 8]), 4, rows.cuda(), 4)
    assert c.scales.view(-1)[3].item() == 2.0 and values(c)[3, :3, 0].tolist() == [448.0, -448.0, 448.0]
    assert ops.device_status(book.ws) == 0


def test_append_and_read_out_of_range(ops):
    book = ops.PageTable.empty(2, 3, 8, 16)
    ops.pages_reserve(book, i32([16, 48]))
    rows = torch.ones(2, 40, 512, dtype=torch.bfloat16, device="cuda")
    for make in (lambda: ops.PagedCache.e4m3(book), lambda: ops.PagedCache.bf16(book, 512)):
        c = make()
        ops.cache_append(c, i32([0, 0]), 4 * 20, rows, 4)    # slot 0 has one page: entries 16..19 are left out
        assert ops.device_status(book.ws) == BOUNDS
        assert int((c.pages.float() != 0).any(-1).sum()) == 16 + 20
        ops.cache_append(c, i32([-1, 0]), 4 * 45, rows, 4)   # 40 rows given, 45 entries asked for
        assert ops.device_status(book.ws) == BOUNDS
        assert int((c.pages.float() != 0).any(-1).sum()) == 16 + 40
        ops.cache_append(c, i32([-1, 4 * 46]), 4 * 5, rows, 4)   # beyond the table
        assert ops.device_status(book.ws) == BOUNDS
        out = ops.cache_read(c, i32([[0, 16, 3], [47, 48, -1]]))
        assert ops.device_status(book.ws) == BOUNDS
        assert (out[0, 0] == 1).all() and (out[0, 1] == 0).all() and (out[0, 2] == 1).all() and (out[1, 1:] == 0).all()


def test_read_past_32_bits(ops):
    """Pages more than 4 GB into a pool."""
    page, num_pages = 64, 150000
    book = ops.PageTable.empty(1, 4, num_pages, page)
    book.table.copy_(i32([[num_pages - 1, 3, 70000, -1]]))
    book.refs[[num_pages - 1, 3, 70000]] = 1
    c = ops.PagedCache.e4m3(book, block=16)
    g = torch.Generator().manual_seed(5)
    rows = torch.randn(1, 192, 512, generator=g).to(torch.bfloat16)
    ops.cache_append(c, i32([0]), 4 * 192, rows.cuda(), 4)
    assert ops.device_status(book.ws) == 0
    out = np64(ops.cache_read(c, torch.arange(192, dtype=torch.int32, device="cuda")[None]))[0]
    codes, scales = np.zeros((3, page, 512)), np.zeros((3, page // 16))
    PO.append(codes, scales, [0, 1, 2], page, 16, 0, 192, np64(rows[0]))
    assert np.array_equal(out, (codes * np.repeat(scales, 16, 1)[..., None]).reshape(192, 512))


# ------------------------------------------------------------------------------------------------ indexer


@pytest.mark.parametrize("page", [16, 64, 128, 512])
@pytest.mark.parametrize("B,S,H_I,pos", [(3, 1, 64, [5, 2047, 1500]), (1, 7, 8, [900]), (2, 5, 128, [2, 1203]), (1, 1, 4, [0])])
def test_indexer_paged(ops, page, B, S, H_I, pos):
    """Bitwise the scores and the selection that the same rows give in a contiguous cache."""
    g = torch.Generator().manual_seed(page + S)
    E = -(-520 // page) * page
    book, table, _ = random_book(ops, g, B, E // page, 2 * B * (E // page), page, [E // page] * B)
    c = ops.PagedCache.bf16(book, 128)
    gg = torch.Generator(device="cuda").manual_seed(S)
    c.pages.normal_(generator=gg)
    q_pos = (i32(pos)[:, None] + torch.arange(S, dtype=torch.int32, device="cuda")).contiguous()
    q = torch.randn(B, S, H_I, 128, generator=gg, device="cuda").to(torch.bfloat16)
    w = torch.randn(B, S, H_I, generator=gg, device="cuda")
    flat = c.pages[book.table.long()].reshape(B, E, 128).contiguous()
    got = ops.indexer_scores_paged(q_pos, q, w, c, scores=torch.full((B, S, E), 9.0, device="cuda"))
    want = ops.indexer_scores(q_pos, q, w, flat, scores=torch.full((B, S, E), 9.0, device="cuda"))
    assert torch.equal(got, want)
    ws = torch.zeros(ops.workspace_size(1, B, S, E, 33), dtype=torch.uint8, device="cuda")
    idx = ops.indexer_topk_paged(q_pos, q, w, c, 33, ws=ws)
    assert torch.equal(idx, ops.indexer_topk(q_pos, q, w, flat, 33))
    assert ops.device_status(ws) == 0
    for b in range(B):
        for i in range(S):
            vis = (int(q_pos[b, i]) + 1) // 4
            if vis:
                check_topk(np64(idx[b, i]), O.indexer_scores(np64(q[b, i]), np64(w[b, i]), np64(flat[b]), vis), 33)


def test_indexer_paged_unmapped(ops):
    """A page that is missing scores 0 and is reported; one behind the visible entries is nobody's business."""
    page, B = 32, 1
    book = ops.PageTable.empty(B, 8, 8, page)
    ops.pages_reserve(book, i32([200]))
    c = ops.PagedCache.bf16(book, 128)
    c.pages.normal_()
    q, w = torch.randn(1, 1, 64, 128, device="cuda").to(torch.bfloat16), torch.randn(1, 1, 64, device="cuda")
    ws = torch.zeros(ops.workspace_size(2, 1, 1, 1, 1), dtype=torch.uint8, device="cuda")
    full = ops.indexer_scores_paged(i32([[799]]), q, w, c, ws=ws).clone()
    assert ops.device_status(ws) == 0
    book.table[0, 2] = -1
    book.table[0, 3] = 99
    got = ops.indexer_scores_paged(i32([[799]]), q, w, c, ws=ws)
    assert ops.device_status(ws) == BOUNDS
    assert (got[0, 0, 64:128] == 0).all()
    keep = [i for i in range(200) if not 64 <= i < 128]
    assert torch.equal(got[0, 0, keep], full[0, 0, keep])


# ------------------------------------------------------------------------------------------------ refusals of the binding


@pytest.mark.parametrize("block", [0, -16, 24, 48, 128])
def test_a_cache_of_another_block_is_refused(ops, block):
    book = ops.PageTable.empty(2, 2, 4, 64)
    with pytest.raises(ValueError):
        ops.PagedCache.e4m3(book, block)


def test_bindings_refuse(ops):
    dev = "cuda"
    book, other = ops.PageTable.empty(2, 4, 8, 16), ops.PageTable.empty(2, 4, 8, 16)
    c8, c16 = ops.PagedCache.e4m3(book, 8), ops.PagedCache.bf16(book, 128)
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device=dev)  # noqa: E731
    bf = torch.bfloat16
    with pytest.raises(TypeError):
        ops.PageTable(z(2, 4, t=torch.int64), z(8), 16)
    with pytest.raises(ValueError):
        ops.PageTable(z(2, 4), z(8), 24)
    with pytest.raises(ValueError):
        ops.PageTable(z(8), z(8), 16)
    for pages, scales in ((z(8, 16, 512, t=bf), z(8, 2, t=torch.float32)), (c8.pages, z(8, 2, t=torch.float64)), (z(8, 16, 128, t=torch.float16), None)):
        with pytest.raises(TypeError):
            ops.PagedCache(book, pages, scales)
    for pages, scales in ((z(7, 16, 128, t=bf), None), (z(8, 32, 128, t=bf), None), (c8.pages, z(8, 3, t=torch.float32)), (c8.pages, z(16, t=torch.float32)),
                          (c8.pages.cpu(), c8.scales)):
        with pytest.raises(ValueError):
            ops.PagedCache(book, pages, scales)
    rows = z(2, 9, 512, t=bf)
    for bad in (dict(start_pos=z(2, 1)), dict(rows=z(3, 9, 512, t=bf)), dict(rows=z(2, 9, 128, t=bf)), dict(rows=z(2, 9, 1024, t=bf)[..., ::2]),
                dict(start_pos=z(2).cpu()), dict(rows=rows.cpu())):
        with pytest.raises(ValueError):
            ops.cache_append(c8, **{**dict(start_pos=z(2), S=4, rows=rows, ratio=4), **bad})
    with pytest.raises(TypeError):
        ops.cache_append(c8, z(2), 4, rows.float(), 4)
    with pytest.raises(ops._lib.CsaError):
        ops.cache_append(c8, z(2), 0, rows, 4)
    with pytest.raises(ops._lib.CsaError):                     # three requests, two slots
        ops.cache_read(c8, z(3, 5))
    for idx, out in ((z(2), None), (z(2, 5), z(2, 5, 128, t=bf))):
        with pytest.raises(ValueError):
            ops.cache_read(c8, idx, out=out)
    with pytest.raises(ValueError):
        ops.pages_reserve(book, z(3))
    with pytest.raises(ValueError):
        ops.pages_fork(book, [ops.PagedCache.bf16(other)], z(2), z(2))
    with pytest.raises(ValueError):
        ops.pages_compact(book, [c8], map=z(7))
    q_idx, w, pos = z(2, 1, 64, 128, t=bf), z(2, 1, 64, t=torch.float32), z(2, 1)
    for cache in (c8, ops.PagedCache.bf16(book, 64)):
        with pytest.raises(ValueError):
            ops.indexer_scores_paged(pos, q_idx, w, cache)
    with pytest.raises(ValueError):
        ops.indexer_topk_paged(pos, q_idx, w, c16, 8, scores=z(2, 1, 63, t=torch.float32))
    q, ring, sink, idx = z(2, 1, 16, 512, t=bf), z(2, 128, 512, t=bf), z(16, t=torch.float32), z(2, 1, 8)
    for bad in (dict(cache=c16), dict(q=z(2, 1, 16, 256, t=bf)), dict(ring=z(1, 128, 512, t=bf)), dict(sink=z(15, t=torch.float32)), dict(topk_idx=z(2, 8)),
                dict(out=z(2, 1, 16, 256, t=bf))):
        with pytest.raises(ValueError):
            ops.sparse_attn8(**{**dict(q_pos=pos, q=q, ring=ring, cache=c8, topk_idx=idx, sink=sink, window=128), **bad})
    with pytest.raises(TypeError):
        ops.hca_attn8(pos, q, ring.float(), c8, sink, 128)
    with pytest.raises(TypeError):
        ops.hca_attn8(pos, q, ring, c8, sink, 128, out=z(2, 1, 16, 512, t=torch.float16))
    for bad in (dict(window=129), dict(window=0), dict(ratio=0), dict(rope_dim=7), dict(scale=float("inf")), dict(ws=z(255, t=torch.uint8))):
        with pytest.raises(ops._lib.CsaError):
            ops.hca_attn8(**{**dict(q_pos=pos, q=q, ring=ring, cache=c8, sink=sink, window=128), **bad})
    assert ops.device_status(book.ws) == 0                      # nothing ran
    assert (c8.pages.view(torch.uint8) == 0).all() and (book.table == -1).all()
