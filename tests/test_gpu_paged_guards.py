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
