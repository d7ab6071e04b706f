"""What the calls on caches in pages refuse or report, beyond arguments out of range."""

import pytest
import torch

pytestmark = pytest.mark.gpu

BOUNDS = 6


@pytest.fixture(scope="module")
def ops():
    from long_context_decode_c4a_b200 import ops
    return ops


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("slots", [4, 2500])   # the slots' arguments in shared memory, in the workspace
@pytest.mark.parametrize("places", [4, 1100])  # one CTA, a cluster
@pytest.mark.parametrize("row,parent,entries,ok", [
    ([0, -1, 1, -1], [0, 0], 40, False),       # a place without a page between two that have one
    ([0, 1, -1, -1], [0, 0], 40, False),       # the partly filled last page
    ([0, 1, -1, -1], [0, 0], 48, False),       # a full last page
    ([-1, -1, -1, -1], [0, 0], 1, False),
    ([0, -1, 1, -1], [-1, 0], 40, False),      # the parent leaves
    ([0, -1, 1, -1], [0, 0], 16, True),        # behind what is taken over
    ([0, -1, 1, -1], [0, 1], 40, True),        # nobody takes it over
    ([0, -1, 1, -1], [-1, 1], 40, True),       # freed
])
def test_fork_of_entries_without_a_page(ops, slots, places, row, parent, entries, ok):
    """Entries that a copy would take over and that have no page: reported, and nothing changes."""
    rows = [row + [-1] * (places - 4)] + [[-1] * places for _ in range(slots - 1)]
    refs = [sum(p == i for p in row) for i in range(2)] + [0] * 6
    book = ops.PageTable(i32(rows), i32(refs), 16)
    cache = ops.PagedCache.bf16(book, 8)
    cache.pages.normal_()
    before = book.table.clone(), book.refs.clone(), cache.pages.clone()
    ops.pages_fork(book, [cache], i32(parent + list(range(2, slots))), i32([entries] + [0] * (slots - 1)))
    assert ops.device_status(book.ws) == (0 if ok else BOUNDS)
    if ok:
        want = [list(row), [-1] * 4]
        want = [want[p][: 4 if p == r else -(-entries // 16)] if p >= 0 else [] for r, p in enumerate(parent)]
        assert book.table[:2, :4].tolist() == [(w + [-1] * 4)[:4] for w in want]
    else:
        for a, b in zip((book.table, book.refs, cache.pages), before):
            assert torch.equal(a, b)


@pytest.mark.parametrize("slots", [3, 700])
@pytest.mark.parametrize("make", [lambda ops, book: ops.PagedCache.e4m3(book, 1), lambda ops, book: ops.PagedCache.e4m3(book, 16),
                                  lambda ops, book: ops.PagedCache.e4m3(book, 32), lambda ops, book: ops.PagedCache.e4m3(book, 64),
                                  lambda ops, book: ops.PagedCache.bf16(book, 512)])
def test_append_to_another_slots_page(ops, make, slots):
    """Rows for a page that another slot has too (a slot rolled back into what it shares) are left out and reported; a page that only
    a holder outside the table has besides takes them."""
    page, last = 64, slots - 1
    rows = [[-1] * 3 for _ in range(slots)]
    rows[0], rows[1], rows[last] = [0, 1, 2], [3, 4, -1], [0, 5, -1] if last > 1 else rows[last]
    refs = [0] * 8
    for row in rows:
        for p in row:
            if p >= 0:
                refs[p] += 1
    refs[4] += 1                                         # a prompt that the caller keeps
    book = ops.PageTable(i32(rows), i32(refs), page)
    cache = make(ops, book)
    g = torch.Generator(device="cuda").manual_seed(1)
    new = torch.randn(2, 192, 512, device="cuda", generator=g).to(torch.bfloat16)
    ops.cache_append(cache, i32([-1, 0]), 60, new, 1)
    assert ops.device_status(book.ws) == 0
    before = cache.pages.float().clone(), None if cache.scales is None else cache.scales.clone()
    ops.cache_append(cache, i32([40, 60]), 60, 100 * new, 1)   # slot 0: entries 40 .. 63 lie on the shared page 0
    assert ops.device_status(book.ws) == BOUNDS
    assert torch.equal(cache.pages[0].float(), before[0][0]) and torch.equal(cache.pages[5].float(), before[0][5])
    if cache.scales is not None:
        assert torch.equal(cache.scales[0], before[1][0])
    got = ops.cache_read(cache, i32([list(range(64, 100)) + [-1] * 24, list(range(60, 120))])).float()
    assert ops.device_status(book.ws) == 0
    # (nearest of four significant bits, subnormals to 2^-10 of a block's step of at most 1 for these rows)
    for b, lo, hi in ((0, 64, 100), (1, 60, 120)):
        x = (100 * new[b, lo:hi]).float()
        assert ((got[b, : hi - lo] - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -9).all()
    ops.cache_append(cache, i32([64, 120]), 8, new, 1)   # slot 0 behind the shared page, slot 1 on the kept one
    assert ops.device_status(book.ws) == 0


def test_handles_keep_their_tensors(ops):
    """The C structs hold the tensors' addresses: another tensor in their place is refused, not forgotten."""
    book = ops.PageTable.empty(2, 4, 8, 16)
    cache = ops.PagedCache.e4m3(book, 8)
    for handle, names in ((book, ("table", "refs", "page_size", "ws", "slots", "max_pages", "num_pages")),
                          (cache, ("pages", "scales", "book", "block", "d"))):
        for name in names:
            held = getattr(handle, name)
            with pytest.raises(AttributeError):
                setattr(handle, name, held.clone() if isinstance(held, torch.Tensor) else held)
            with pytest.raises(AttributeError):
                delattr(handle, name)
            assert getattr(handle, name) is held
    book.table[0, 0] = 3                                 # their contents are the caller's
    cache.scales.fill_(1.0)
